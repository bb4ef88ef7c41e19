"""The operators of a decoding step with drafted tokens: cases, their plain form in
elementary torch operations, and the library's calls.

Kinds of cases:

  tree     attention of the nodes of a tree of drafted tokens over the paged cache
  verify   which drafted tokens the target model accepts, and the token after them, from
           given random numbers
  keep     the accepted nodes' cache rows moved together, in every layer

A tree of request r has n <= Tn nodes; parents[r, i] < i, -1 for a root.  Node i's key and
value are cached behind the request's seq_lens[r] tokens, at position seq_lens[r] + i; it
sees those tokens, its ancestors and itself.
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
        # the 64-request decode workload with a small tree for each request
        dict(name="tree_64req_8", kind="tree", S=64, Tn=8, Hq=12, Hkv=2, D=128, lo=512, hi=8192,
             chain=False, ragged=False, lens=5003),
        # 16 requests of a grouped-query model with wide trees
        dict(name="tree_16req_64", kind="tree", S=16, Tn=64, Hq=32, Hkv=8, D=128, lo=1024, hi=8192,
             chain=False, ragged=True, lens=6003),
        # one long conversation
        dict(name="tree_1x128k", kind="tree", S=1, Tn=32, Hq=32, Hkv=8, D=128, lo=131000,
             hi=131000, chain=False, ragged=False, lens=5005),
        # a chain of five tokens for one request that has just begun: latency counts
        dict(name="tree_small_chain", kind="tree", S=1, Tn=5, Hq=8, Hkv=2, D=64, lo=100, hi=300,
             chain=True, ragged=False, lens=5006),
        # a few requests of unlike length and tree, narrow heads, odd sizes
        dict(name="tree_odd_d64", kind="tree", S=7, Tn=37, Hq=9, Hkv=3, D=64, lo=0, hi=1500,
             chain=False, ragged=True, lens=6005),
        # the widest trees: many rows share the cache, arithmetic counts
        dict(name="tree_wide_200", kind="tree", S=8, Tn=200, Hq=32, Hkv=4, D=128, lo=2000, hi=16000,
             chain=False, ragged=False, lens=5007),
        # a drafted chain of one request, a small vocabulary: latency counts
        dict(name="verify_1x8", kind="verify", S=1, Tn=8, V=32000, chain=True, ragged=False,
             drawn=True, lens=5008),
        # the 64 requests' trees, children drawn from the draft's probabilities
        dict(name="verify_64x8", kind="verify", S=64, Tn=8, V=131072, chain=False, ragged=False,
             drawn=True, lens=5003),
        # trees of the draft's likeliest tokens, an odd vocabulary
        dict(name="verify_16x24_top", kind="verify", S=16, Tn=24, V=50021, chain=False, ragged=True,
             drawn=False, lens=6003),
        # more requests with longer chains
        dict(name="verify_128x5", kind="verify", S=128, Tn=5, V=100003, chain=True, ragged=False,
             drawn=True, lens=6006),
        # one layer's cache of a few requests
        dict(name="keep_4x1", kind="keep", S=4, Tn=16, Hkv=2, D=128, layers=1, lo=0, hi=500,
             chain=False, ragged=False, lens=5009),
        # the caches of all layers of a model
        dict(name="keep_64x32", kind="keep", S=64, Tn=32, Hkv=8, D=128, layers=32, lo=16, hi=300,
             chain=False, ragged=True, lens=5010),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["tree", "tree", "tree", "verify", "verify", "keep"])
    c = dict(kind=kind, Tn=_log(rng, 1, 256 if kind == "tree" else 64),
             chain=rng.random() < 0.3, ragged=rng.random() < 0.5, lens=rng.randrange(1 << 30))
    if kind == "verify":
        V = _log(rng, 500, 160000)
        if c["Tn"] > 16 and not c["chain"]:
            c["Tn"] //= 2
        c |= dict(S=max(1, min(_log(rng, 1, 200), (1 << 26) // (V * c["Tn"]))), V=V,
                  drawn=rng.random() < 0.6)
        return c
    D = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    c |= dict(Hkv=Hkv, D=D)
    if kind == "keep":
        hi = _log(rng, 1, 1000)
        c |= dict(lo=rng.choice([0, hi]), hi=hi, layers=_log(rng, 1, 40))
        c["S"] = max(1, min(_log(rng, 1, 100), 500000 // ((hi + c["Tn"]) * Hkv * c["layers"])))
        return c
    Hq = Hkv * rng.choice([1, 2, 3, 4, 6, 8, 16])
    while Hq > 48:
        Hq //= 2
        Hq -= Hq % Hkv
    hi = _log(rng, 1, 60000)
    while c["Tn"] * hi * Hq * D > 4 * 10 ** 10:
        hi //= 2
    S = min(_log(rng, 1, 100), 1000000 // (hi * Hkv), 4 * 10 ** 10 // (c["Tn"] * hi * Hq * D))
    return c | dict(S=max(1, S), Hq=Hq, lo=min(hi, rng.choice([0, 1, hi // 8])), hi=hi)


def _sizes(c):
    """Tokens cached before the tree, and the nodes of the tree, of each request."""
    rng = random.Random(c["lens"])
    lens = [rng.randint(c.get("lo", 0), c.get("hi", 0)) for _ in range(c["S"])]
    nodes = [rng.randint(0, c["Tn"]) if c["ragged"] else c["Tn"] for _ in range(c["S"])]
    return lens, nodes


def _paths(c):
    """Accepted nodes of each request: the first few, then some far down the tree (behind all
    the rows that are written, so that a pass may be repeated)."""
    rng = random.Random(c["lens"] + 1)
    paths = []
    for n in _sizes(c)[1]:
        m = min(n, 1 + min(int(rng.expovariate(0.35)), 12))
        near = m if c["chain"] or m == 0 else rng.randint(1, m)
        far = min(m - near, n - m)
        paths.append(list(range(near)) + sorted(rng.sample(range(m, n), far)))
    return paths


# --------------------------------------------------------------------------- #
# inputs
# --------------------------------------------------------------------------- #
def _parents(c, gen):
    """A random tree for each request: earlier nodes have more children."""
    S, Tn = c["S"], c["Tn"]
    i = torch.arange(Tn, device="cuda")
    if c["chain"]:
        return (i - 1).int().expand(S, Tn).contiguous()
    u = torch.rand(S, Tn, generator=gen, device="cuda")
    p = (i * u ** 1.5).floor().int().minimum(i.int() - 1)
    p[:, 0] = -1
    return p


def _table(c, lens, gen):
    """Block table (a random permutation of the pool), and the pool's number of blocks."""
    blocks = torch.tensor([-(-(n + c["Tn"]) // BS) for n in lens])
    used = int(blocks.sum())
    NB = used + -(-used // 8)
    perm = torch.randperm(NB, generator=gen, device="cuda").int()
    col = torch.arange(int(blocks.max()))[None, :]
    index = (blocks.cumsum(0) - blocks)[:, None] + col
    live = (col < blocks[:, None]).cuda()
    return torch.where(live, perm[index.clamp(max=NB - 1).cuda()], -1), NB


def _probabilities(c, st, gen):
    """The target's and the draft's distributions, like enough that drafts are often accepted,
    and drafted tokens: drawn from the parent's row, or its likeliest tokens in turn."""
    S, Tn, V = c["S"], c["Tn"], c["V"]
    logits = 3 * torch.randn(S, Tn, V, generator=gen, device="cuda")
    st["p"] = logits.softmax(-1)
    logits += 0.6 * torch.randn(S, Tn, V, generator=gen, device="cuda")
    parent = st["parents"].long().clamp(min=0)
    if c["drawn"]:
        st["q"] = logits.softmax(-1)
        # the largest of probability / exponential is a draw
        race = torch.empty(S, V, device="cuda")
        st["tokens"] = torch.empty(S, Tn, dtype=torch.int32, device="cuda")
        rows = torch.arange(S, device="cuda")
        for i in range(Tn):
            race.exponential_(generator=gen)
            st["tokens"][:, i] = (st["q"][rows, parent[:, i]] / race).argmax(-1)
    else:
        st["q"] = None
        same = (parent[:, :, None] == parent[:, None, :]).tril(-1)
        same[:, :, 0] = False
        rank = same.sum(-1)  # of a node among its siblings
        top = logits.topk(min(V, int(rank.max()) + 1), -1).indices
        top = top.gather(1, parent[:, :, None].expand(-1, -1, top.shape[-1]))
        st["tokens"] = top.gather(2, rank[:, :, None])[:, :, 0].int()
    st["u"] = torch.rand(S, Tn, generator=gen, device="cuda")


def prepare(case, seed):
    c = case
    gen = torch.Generator("cuda").manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    st = dict(c)
    S, Tn = c["S"], c["Tn"]
    lens, nodes = _sizes(c)
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    st["nodes"] = torch.tensor(nodes, dtype=torch.int32, device="cuda") if c["ragged"] else None
    st["parents"] = _parents(c, gen)
    if c["kind"] == "verify":
        _probabilities(c, st, gen)
        return st
    Hkv, D = c["Hkv"], c["D"]
    st["table"], NB = _table(c, lens, gen)
    if c["kind"] == "tree":
        gain = torch.exp(0.3 * randn(2, Hkv, 1, D))
        st["kp"], st["vp"] = ((randn(NB, Hkv, BS, D) * gain[i]).bfloat16() for i in (0, 1))
        st["q"] = randn(S, c["Hq"], Tn, D).bfloat16()
        st["max_len"] = max(lens) + Tn
        return st
    paths = _paths(c)
    st["counts"] = torch.tensor([len(p) for p in paths], dtype=torch.int32, device="cuda")
    st["path"] = torch.tensor([p + [-1] * (Tn - len(p)) for p in paths], dtype=torch.int32,
                              device="cuda")
    # the pools of all layers
    st["kps"], st["vps"] = (torch.empty(c["layers"], NB, Hkv, BS, D, dtype=torch.bfloat16,
                                        device="cuda").normal_(generator=gen) for _ in (0, 1))
    st["new"] = torch.empty_like(st["lens"])
    return st


# --------------------------------------------------------------------------- #
# the plain form
# --------------------------------------------------------------------------- #
def _ancestors(parents):
    """[S, Tn, Tn]: whether node j is node i or one of its ancestors."""
    S, Tn = parents.shape
    i = torch.arange(Tn, device=parents.device)
    up = i.expand(S, Tn)
    seen = torch.zeros(S, Tn, Tn + 1, dtype=torch.bool, device=parents.device)
    above = torch.cat([parents.long(), torch.full((S, 1), -1, device=parents.device)], 1)
    for _ in range(Tn):
        seen.scatter_(2, torch.where(up < 0, Tn, up)[:, :, None], True)
        up = above.gather(1, torch.where(up < 0, Tn, up))
    return seen[:, :, :Tn]


def _plain_tree(st):
    S, Hq, Hkv, Tn, D = (st[x] for x in ("S", "Hq", "Hkv", "Tn", "D"))
    n = st["nodes"].long() if st["nodes"] is not None else torch.full((S,), Tn, device="cuda")
    t = torch.arange(st["max_len"], device="cuda")
    blk = st["table"].long()[:, t // BS].clamp(min=0)
    k, v = (pool[blk, :, t % BS].transpose(1, 2).float() for pool in (st["kp"], st["vp"]))
    # [S, Tn, max_len]: the cached tokens, then the node's ancestors
    at = t - st["lens"].long()[:, None]
    anc = _ancestors(st["parents"])
    seen = anc.gather(2, at.clamp(0, Tn - 1)[:, None].expand(S, Tn, -1))
    mask = (at < 0)[:, None] | (seen & (at < Tn)[:, None])
    mask &= (torch.arange(Tn, device="cuda") < n[:, None])[:, :, None]
    # the heads of a KV head as rows
    s = (st["q"].float().reshape(S, Hkv, -1, D) @ k.transpose(2, 3)) * (1 / math.sqrt(D))
    s = s.view(S, Hq, Tn, -1).masked_fill_(~mask[:, None], -torch.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp_(s.sub_(torch.where(m.isfinite(), m, 0.0)))
    l = p.sum(-1, keepdim=True)
    o = (p.view(S, Hkv, -1, p.shape[-1]) @ v).view(S, Hq, Tn, D) / torch.where(l > 0, l, 1.0)
    return [o.bfloat16(), (m + torch.log(l)).squeeze(-1)]


def _plain_verify(st):
    """Node after node, every request at once; probabilities in 64 bits, as an accepted token
    hangs on which side of a border a random number lies."""
    S, Tn, V = st["S"], st["Tn"], st["V"]
    rows = torch.arange(S, device="cuda")
    n = st["nodes"].long() if st["nodes"] is not None else torch.full((S,), Tn, device="cuda")
    tokens, parents, u = st["tokens"].long(), st["parents"].long(), st["u"].double()
    cur = torch.zeros(S, dtype=torch.long, device="cuda")
    w, total = st["p"][:, 0].double(), torch.ones(S, dtype=torch.float64, device="cuda")
    path = torch.full((S, Tn), -1, dtype=torch.int32, device="cuda")
    out = torch.full((S, Tn), -1, dtype=torch.int32, device="cuda")
    path[:, 0] = torch.where(n > 0, 0, -1)
    count = (n > 0).long()
    for i in range(1, Tn):
        tested = (parents[:, i] == cur) & (i < n)
        x = tokens[:, i:i + 1]
        if st["q"] is not None:
            q = st["q"][rows, cur].double()
        else:
            q = torch.zeros_like(w).scatter_(1, x, 1.0)
        accepted = tested & (u[:, i] * q.gather(1, x)[:, 0] * total < w.gather(1, x)[:, 0])
        rest = (w - q * total[:, None]).clamp_(min=0)
        mass = rest.sum(1)
        rejected = tested & ~accepted & (mass > 0)
        at = count.clamp(max=Tn - 1)
        path[rows, at] = torch.where(accepted, i, path[rows, at])
        out[rows, at - 1] = torch.where(accepted, x[:, 0].int(), out[rows, at - 1])
        cur = torch.where(accepted, i, cur)
        count = count + accepted
        w = torch.where(accepted[:, None], st["p"][:, i].double(),
                        torch.where(rejected[:, None], rest, w))
        total = torch.where(accepted, 1.0, torch.where(rejected, mass, total))
    c = w.cumsum(1)
    last = (c <= u[:, :1] * c[:, -1:]).sum(1)
    last = torch.where(last < V, last, -1)
    at = (count - 1).clamp(min=0)
    out[rows, at] = torch.where(n > 0, last.int(), out[rows, at])
    return [out, path, count.int()]


def _plain_keep(st):
    j = torch.arange(st["Tn"], device="cuda")
    r, j = torch.nonzero(j < st["counts"][:, None], as_tuple=True)
    dst = st["lens"].long()[r] + j
    src = st["lens"].long()[r] + st["path"].long()[r, j]
    table = st["table"].long()
    for pool in (st["kps"], st["vps"]):
        pool[:, table[r, dst // BS], :, dst % BS] = pool[:, table[r, src // BS], :, src % BS]
    st["new"].copy_(st["lens"] + st["counts"])
    return [st["new"], st["kps"], st["vps"]]


# --------------------------------------------------------------------------- #
# the library's calls
# --------------------------------------------------------------------------- #
def _calls(st):
    import attention_flashattention_fwd_03_gb300 as gb

    if st["kind"] == "tree":
        return list(gb.paged_attn_tree(st["q"], st["kp"], st["vp"], st["table"], st["lens"],
                                       st["parents"], st["max_len"], tree_lens=st["nodes"]))
    if st["kind"] == "verify":
        return list(gb.draft_verify(st["p"], st["q"], st["tokens"], st["parents"], st["u"],
                                    tree_lens=st["nodes"]))
    gb.paged_kv_keep(st["kps"], st["vps"], st["table"], st["lens"], st["path"], st["counts"],
                     new_seq_lens=st["new"])
    return [st["new"], st["kps"], st["vps"]]


def run(state):
    if own:
        return _calls(state)
    return {"tree": _plain_tree, "verify": _plain_verify, "keep": _plain_keep}[state["kind"]](state)


# --------------------------------------------------------------------------- #
# what a pass cannot do without
# --------------------------------------------------------------------------- #
def work(case):
    c = case
    lens, nodes = _sizes(c)
    S, Tn = c["S"], c["Tn"]
    if c["kind"] == "verify":
        # one row of each distribution to draw the last token from; what is tested is single values
        rows = sum(n > 0 for n in nodes)
        return {"bytes": rows * c["V"] * (8 if c["drawn"] else 4) + S * Tn * 20,
                "flops": rows * c["V"] * (4 if c["drawn"] else 1)}
    if c["kind"] == "keep":
        moved = sum(i != j for p in _paths(c) for j, i in enumerate(p))
        return {"bytes": moved * c["layers"] * c["Hkv"] * c["D"] * 8 + S * (12 + Tn * 4), "flops": 0}
    # (every node sees the cached tokens and itself at least)
    pairs = sum(n * (L + 1) for L, n in zip(lens, nodes))
    keys = sum(L + n for L, n in zip(lens, nodes))
    return {"bytes": S * Tn * c["Hq"] * (4 * c["D"] + 4) + keys * c["Hkv"] * c["D"] * 4 +
                     keys // BS * 4 + S * (8 + 4 * Tn),
            "flops": 4 * c["D"] * c["Hq"] * pairs}


# --------------------------------------------------------------------------- #
# the definition in 64 bits
# --------------------------------------------------------------------------- #
def _exact_tree(c, st):
    lens, nodes = _sizes(c)
    Hq, Hkv, Tn, D = c["Hq"], c["Hkv"], c["Tn"], c["D"]
    o = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(st["q"].shape[:-1], -torch.inf, dtype=torch.float64, device="cuda")
    parents = st["parents"].tolist()
    for r, (L, n) in enumerate(zip(lens, nodes)):
        if n == 0:
            continue
        hidden = torch.ones(n, n, dtype=torch.bool)
        for i in range(n):
            a = i
            while a >= 0:
                hidden[i, a] = False
                a = parents[r][a]
        hidden = torch.cat([torch.zeros(n, L, dtype=torch.bool), hidden], 1).cuda()
        blocks = st["table"][r, :-(-(L + n) // BS)].long()
        for h in range(Hkv):
            k, v = (x[blocks, h].reshape(-1, D)[:L + n].double() for x in (st["kp"], st["vp"]))
            for g in range(h * (Hq // Hkv), (h + 1) * (Hq // Hkv)):
                s = st["q"][r, g, :n].double() @ k.T / math.sqrt(D)
                s[hidden] = -torch.inf
                lse[r, g, :n] = torch.logsumexp(s, 1)
                o[r, g, :n] = torch.softmax(s, 1) @ v
    return [o, lse]


def _exact_verify(c, st):
    """Request after request, with residual distributions that are normalised each time."""
    nodes = _sizes(c)[1]
    Tn, V = c["Tn"], c["V"]
    tokens, parents = st["tokens"].tolist(), st["parents"].tolist()
    out, path = ([[-1] * Tn for _ in nodes] for _ in (0, 1))
    counts = []
    for r, n in enumerate(nodes):
        if n == 0:
            counts.append(0)
            continue
        u = st["u"][r].double().tolist()
        cur, kept, said = 0, [0], []
        dist = st["p"][r, 0].double()
        for i in range(1, n):
            if parents[r][i] != cur:
                continue
            x = tokens[r][i]
            if st["q"] is None:
                draft = torch.zeros(V, dtype=torch.float64, device="cuda")
                draft[x] = 1
            else:
                draft = st["q"][r, cur].double()
            if u[i] * float(draft[x]) < float(dist[x]):
                cur = i
                kept.append(i)
                said.append(x)
                dist = st["p"][r, i].double()
                continue
            rest = torch.relu(dist - draft)
            if float(rest.sum()) > 0:
                dist = rest / rest.sum()
        last = int(torch.searchsorted(dist.cumsum(0), u[0] * float(dist.sum()), right=True))
        said.append(last if last < V else -1)
        path[r][:len(kept)], out[r][:len(said)] = kept, said
        counts.append(len(kept))
    return [torch.tensor(x, dtype=torch.int32, device="cuda") for x in (out, path, counts)]


def _exact_keep(c, st):
    lens, paths = _sizes(c)[0], _paths(c)
    new = torch.tensor([L + len(p) for L, p in zip(lens, paths)], dtype=torch.int32, device="cuda")
    table = st["table"].tolist()
    moves = [(table[r][(lens[r] + i) // BS] * BS + (lens[r] + i) % BS,
              table[r][(lens[r] + j) // BS] * BS + (lens[r] + j) % BS)
             for r, p in enumerate(paths) for j, i in enumerate(p) if i != j]
    src, dst = (torch.tensor(x, dtype=torch.long, device="cuda") for x in zip(*moves)) if moves else \
        (torch.zeros(0, dtype=torch.long, device="cuda"),) * 2
    pools = []
    for stacked in (st["kps"], st["vps"]):
        moved = stacked.double()
        for layer in moved:
            rows = layer.transpose(1, 2).reshape(-1, c["Hkv"], c["D"])  # [token slot, head, channel]
            rows[dst] = rows[src]
            layer.copy_(rows.view(-1, BS, c["Hkv"], c["D"]).transpose(1, 2))
        pools.append(moved)
    return [new, *pools]


def exact(case, seed):
    st = prepare(case, seed)
    return {"tree": _exact_tree, "verify": _exact_verify, "keep": _exact_keep}[case["kind"]](case, st)
