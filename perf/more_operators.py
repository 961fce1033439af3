"""The operators of speculative decoding over a paged bf16 key/value cache, as they are measured:
attention for the trees of drafted tokens, their verification against the target's
probabilities, and keeping the accepted tokens' rows of the cache.

A cache is, per layer, bf16 [num_pages, Hkv, page_size, d] for the keys and for the values;
sequence b's token j lives in page block_table[b, j // page_size], row j % page_size.  A tree of
up to Nt drafted tokens per sequence is given by each node's parent, an earlier node (-1: a node
without a parent in the tree; -2: no node, where sequences draft fewer tokens than others), and
node j of sequence b is its token seq_lens[b] + j.

``own`` selects the framework's calls; otherwise every operator runs in its plain form,
elementary torch operations in 32 bits (verification in 64, where values lie next to a border).
``exact`` restates the attention in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------- the cases

def listed():
    return [
        # one chat turn of a single user, sixteen drafted tokens: latency
        dict(name="tree one short sequence", op="tree", B=1, H=32, Hkv=8, Nt=16, Nq=16, d=128, page=16,
             lo=1000, hi=1000, chain=False, ragged=False),
        # drafting itself: the newest level of a growing tree, eight of its 24 nodes
        dict(name="tree newest level", op="tree", B=4, H=16, Hkv=4, Nt=24, Nq=8, d=96, page=16, lo=300,
             hi=2500, chain=False, ragged=False),
        # continuous batching: every sequence at another length, with another number of drafts
        dict(name="tree ragged batch", op="tree", B=32, H=32, Hkv=8, Nt=32, Nq=32, d=128, page=64, lo=1,
             hi=8192, chain=False, ragged=True),
        # a long document and a wide tree: one sequence has to fill the GPU
        dict(name="tree one long sequence", op="tree", B=1, H=32, Hkv=8, Nt=64, Nq=64, d=128, page=16,
             lo=131072, hi=131072, chain=False, ragged=False),
        # four tokens drafted in a row, no branches
        dict(name="tree chain of four", op="tree", B=8, H=32, Hkv=4, Nt=4, Nq=4, d=64, page=32, lo=5000,
             hi=32768, chain=True, ragged=False),
        # wide heads, pages whose size is no power of two
        dict(name="tree wide heads odd pages", op="tree", B=5, H=16, Hkv=2, Nt=21, Nq=21, d=256, page=48,
             lo=101, hi=2899, chain=False, ragged=True),
        # many queries per key: products, not the cache's bytes, are what it has to do
        dict(name="tree large batch", op="tree", B=16, H=64, Hkv=8, Nt=48, Nq=48, d=128, page=64, lo=16384,
             hi=32768, chain=False, ragged=False),
        # a single user's drafts: latency of the walk down the tree
        dict(name="verify one sequence", op="verify", B=1, Nt=16, V=32000, dtype="float32", draft="probs",
             replacement=True, ragged=False),
        # a server's step: many sequences, a large vocabulary, drafts without repetition
        dict(name="verify batch", op="verify", B=64, Nt=24, V=128000, dtype="float32", draft="probs",
             replacement=False, ragged=True),
        # drafts that were looked up instead of drawn, an odd vocabulary, 16-bit probabilities
        dict(name="verify looked up drafts", op="verify", B=48, Nt=9, V=50021, dtype="bfloat16", draft="none",
             replacement=True, ragged=True),
        # the accepted tokens of one user in every layer of a model
        dict(name="keep one sequence", op="keep", B=1, Hkv=8, d=128, page=16, Nt=16, lo=1000, hi=1000,
             layers=24),
        # the accepted tokens of a large batch
        dict(name="keep batch", op="keep", B=64, Hkv=8, d=128, page=32, Nt=32, lo=1, hi=600, layers=24),
    ]


def _log_int(rng, lo, hi):
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    op = rng.choice(("tree", "tree", "tree", "verify", "keep"))
    page = rng.choice((8, 16, 24, 32, 48, 64, 128))
    d = rng.choice((64, 96, 128, 256))
    if op == "tree":
        Hkv = rng.choice((1, 2, 4, 5, 8, 16))
        G = rng.choice((1, 2, 3, 4, 6, 8))
        B, Nt = _log_int(rng, 1, 64), _log_int(rng, 1, 128)
        chain = rng.random() < 0.2
        Nq = Nt if chain else rng.choice((Nt, Nt, rng.randint(1, Nt)))
        most = min(300_000_000 // (B * Hkv * d), 50_000_000_000 // (B * Hkv * G * Nq * d))
        hi = _log_int(rng, 20, max(21, min(100000, most)))
        return dict(op=op, B=B, H=Hkv * G, Hkv=Hkv, Nt=Nt, Nq=Nq, d=d, page=page,
                    lo=rng.choice((0, hi // 3 + 1, hi)), hi=hi, chain=chain,
                    ragged=rng.random() < 0.5)
    if op == "verify":
        V = _log_int(rng, 1000, 160000)
        Nt = _log_int(rng, 2, 48)
        B = _log_int(rng, 1, max(1, min(150, 180_000_000 // (V * Nt))))
        return dict(op=op, B=B, Nt=Nt, V=V, dtype=rng.choice(("float32", "float32", "bfloat16")),
                    draft=rng.choice(("probs", "probs", "none")), replacement=rng.random() < 0.5,
                    ragged=rng.random() < 0.5)
    B, Hkv, Nt = _log_int(rng, 1, 100), rng.choice((1, 2, 4, 8)), rng.randint(1, 64)
    hi = _log_int(rng, 1, 500)
    return dict(op=op, B=B, Hkv=Hkv, d=d, page=page, Nt=Nt, lo=rng.choice((0, hi)), hi=hi,
                layers=rng.choice((1, 2, 5, 16)))


def _lens(B, lo, hi):
    """B lengths spread over lo..hi, the same for every seed."""
    return [lo + int((hi - lo + 1) * ((b + 1) * 0.6180339887498949 % 1.0)) for b in range(B)]


# ------------------------------------------------------------------ the inputs

def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _paged(g, lens, page):
    """Block table of sequences of these lengths, their pages scattered over a cache of num_pages."""
    need = [-(-n // page) for n in lens]
    num_pages = sum(need) + max(3, sum(need) // 16)
    width = max(1, max(need))
    perm = torch.randperm(num_pages, generator=g, device=DEV)[:sum(need)].to(torch.int32)
    table = torch.zeros((len(lens), width), dtype=torch.int32, device=DEV)
    used = torch.arange(width, device=DEV)[None] < torch.tensor(need, device=DEV)[:, None]
    table[used] = perm
    return table, num_pages


def _parents(g, B, Nt, ragged):
    """Trees under node 0 with more children near the root; ragged: of different sizes, a sequence's
    last places empty."""
    j = torch.arange(Nt, device=DEV)
    u = torch.rand((B, Nt), generator=g, device=DEV)
    parents = torch.where(j > 0, (u * u * j).long().clamp(max=Nt - 1), -1)
    parents = torch.minimum(parents, j - 1)
    if ragged:
        size = 1 + (torch.rand((B, 1), generator=g, device=DEV) * Nt).long().clamp(max=Nt - 1)
        parents = torch.where(j < size, parents, -2)
    return parents.to(torch.int32)


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16)


def prepare(case, seed):
    c, g = case, _generator(seed)
    if c["op"] == "verify":
        return _prepare_verify(c, g)
    lens = _lens(c["B"], c["lo"], c["hi"])
    table, num_pages = _paged(g, [n + c["Nt"] for n in lens], c["page"])
    shape = (num_pages, c["Hkv"], c["page"], c["d"])
    s = dict(op=c["op"], table=table, lens=torch.tensor(lens, dtype=torch.int32, device=DEV), Nt=c["Nt"])
    if c["op"] == "tree":
        s["parents"] = None if c["chain"] else _parents(g, c["B"], c["Nt"], c["ragged"])
        s["q"] = _normal(g, c["B"], c["H"], c["Nq"], c["d"])
        s["k_cache"], s["v_cache"] = _normal(g, *shape), _normal(g, *shape)
        return s
    s["caches"] = [_normal(g, *shape) for _ in range(2 * c["layers"])]
    # accepted paths: node 0 and about every third of what follows, as deep as drafts are good
    B, Nt = c["B"], c["Nt"]
    take = torch.rand((B, Nt), generator=g, device=DEV) < 0.3
    take[:, 0] = True
    take &= take.cumsum(1) <= 1 + (torch.rand((B, 1), generator=g, device=DEV) * 8).long()
    node = torch.where(take, torch.arange(Nt, device=DEV), Nt).sort(1).values
    s["path"] = torch.where(node < Nt, node, -1).to(torch.int32)
    s["count"] = take.sum(1, dtype=torch.int32)
    return s


def _prepare_verify(c, g):
    """The target's probabilities after every node, a draft's that resemble them, drafted tokens
    drawn from the draft's at their parents (or, looked up, the target's likeliest or another)."""
    B, Nt, V = c["B"], c["Nt"], c["V"]
    dtype = getattr(torch, c["dtype"])
    parents = _parents(g, B, Nt, c["ragged"])
    target = torch.empty((B, Nt, V), dtype=dtype, device=DEV)
    draft = torch.empty_like(target) if c["draft"] == "probs" else None
    tokens = torch.zeros((B, Nt), dtype=torch.int64, device=DEV)
    for b in range(B):
        x = 3 * torch.randn((Nt, V), generator=g, device=DEV)
        p = torch.softmax(x, -1)
        target[b] = p
        up = parents[b].clamp(min=0).long()
        if draft is None:
            top = p.topk(min(4, V), -1).indices[up]
            pick = torch.randint(top.shape[1], (Nt, 1), generator=g, device=DEV)
            tokens[b] = top.gather(1, pick).squeeze(1)
        else:
            q = torch.softmax(x + 0.7 * torch.randn((Nt, V), generator=g, device=DEV), -1)
            draft[b] = q
            if c["replacement"]:
                tokens[b] = torch.multinomial(q[up], 1, generator=g).squeeze(1)
            else:
                # a parent's children without repetition: the first of its draws that none took
                order = torch.multinomial(q, min(Nt, V), generator=g)
                j = torch.arange(Nt, device=DEV)
                older = ((up[None] == up[:, None]) & (j[None] < j[:, None]) & (j[None] > 0)).sum(1)
                tokens[b] = order[up, older]
    tokens = tokens.to(torch.int32)
    uniform = torch.rand((B, Nt), generator=g, device=DEV)
    return dict(op="verify", tokens=tokens, parents=parents, target=target, draft=draft, uniform=uniform,
                replacement=c["replacement"])


# ---------------------------------------------------------------- one pass

def run(state):
    s = state
    if own:
        import exact_attention_26_gb300 as fa
        if s["op"] == "tree":
            return fa.decode_paged_tree(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["parents"])
        if s["op"] == "verify":
            return fa.verify_tree(s["tokens"], s["parents"], s["target"], s["draft"], s["uniform"],
                                  replacement=s["replacement"])
        lens = fa.keep_path(s["caches"], s["table"], s["lens"], s["path"], s["count"])
        return [lens, *s["caches"]]
    if s["op"] == "tree":
        return _plain_tree(s)
    if s["op"] == "verify":
        return _plain_verify(s)
    return [_plain_keep(s), *s["caches"]]


def _plain_tree(s):
    q, table, lens = s["q"], s["table"].long(), s["lens"].long()
    B, H, Nq, d = q.shape
    _, Hkv, page, _ = s["k_cache"].shape
    width, Nt = table.shape[1], s["Nt"]
    keys = width * page

    def gather(cache):  # [B, Hkv, keys, d], 32 bits
        return cache[table].float().transpose(1, 2).reshape(B, Hkv, keys, d)

    x = (q.float().reshape(B, Hkv, -1, d) @ gather(s["k_cache"]).transpose(2, 3)) / math.sqrt(d)
    x = x.reshape(B, H, Nq, keys)
    # which nodes a node sees: itself and its ancestors, by repeated squaring of "itself or parent"
    j = torch.arange(Nt, device=DEV)
    parents = s["parents"] if s["parents"] is not None else (j - 1)[None].expand(B, Nt)
    here = parents >= -1
    see = ((parents[:, :, None] == j) | (j[:, None] == j)).float()
    for _ in range(max(1, Nt - 1).bit_length()):
        see = (see @ see > 0).float()
    see = (see > 0) & here[:, :, None]
    node = torch.arange(keys, device=DEV)[None] - lens[:, None]  # which node a key is
    tree = see[:, Nt - Nq:].gather(2, node.clamp(0, Nt - 1)[:, None].expand(B, Nq, keys))
    seen = (node < 0)[:, None] & here[:, Nt - Nq:, None] | ((node >= 0) & (node < Nt))[:, None] & tree
    x = torch.where(seen[:, None], x, -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    o = (p.reshape(B, Hkv, -1, keys) @ gather(s["v_cache"])).reshape(B, H, Nq, d)
    o = torch.where(total > 0, o / total, 0.0)
    return o.to(torch.bfloat16), (m + torch.log(total)).squeeze(-1)


def _plain_verify(s):
    """The walk down every tree at once, node by node in order: a node is tried when the walk
    stands at its parent.  Behind the k-th rejection at a node the token is to be drawn from what
    the drafts tried so far leave of the target's probabilities, max(p - a q, 0) over its sum."""
    parents, tokens, u = s["parents"].long(), s["tokens"].long(), s["uniform"].double()
    target, draft = s["target"], s["draft"]
    B, Nt, V = target.shape
    rows = torch.arange(B, device=DEV)
    cur = torch.zeros(B, dtype=torch.long, device=DEV)
    path = torch.full((B, Nt + 1), -1, dtype=torch.long, device=DEV)
    path[:, 0] = 0
    count = torch.ones(B, dtype=torch.long, device=DEV)
    a = torch.zeros(B, dtype=torch.float64, device=DEV)      # of the draft's probabilities, to take off
    used = torch.zeros_like(a)                               # draft's probability of the rejected tokens
    total = torch.ones_like(a)
    gone = torch.zeros((B, V + 1), dtype=torch.bool, device=DEV)  # looked up drafts that were rejected

    def left(cur, a, gone):
        p = target[rows, cur].double()
        if draft is None:
            return torch.where(gone[:, :V], 0.0, p)
        return (p - a[:, None] * draft[rows, cur].double()).clamp(min=0.0)

    for j in range(1, Nt):
        tried = parents[:, j] == cur
        x = tokens[:, j]
        px = target[rows, cur, x].double()
        if draft is None:
            wx, qx = torch.where(gone[rows, x], 0.0, px), torch.ones_like(a)
        else:
            qx = draft[rows, cur, x].double()
            wx = (px - a * qx).clamp(min=0.0)
        rest = torch.ones_like(a) if s["replacement"] else (1.0 - used).clamp(min=2.0 ** -60)
        yes = tried & (u[:, j] * (qx / rest) * total < wx)
        no = tried & ~yes
        if draft is None:
            gone[rows, torch.where(no, x, V)] = True
            total = torch.where(no, total - wx, total)
        else:
            a = torch.where(no, (a + total / rest).clamp(max=2.0 ** 60), a)
            used = torch.where(no, used + qx, used)
            total = torch.where(no, left(cur, a, gone).sum(-1), total)
        cur = torch.where(yes, j, cur)
        path[rows, torch.where(yes, count, Nt)] = torch.where(yes, j, -1)
        count = count + yes
        a, used = torch.where(yes, 0.0, a), torch.where(yes, 0.0, used)
        total = torch.where(yes, 1.0, total)
        gone = gone & ~yes[:, None]
    w = left(cur, a, gone)
    w = torch.where((w.sum(-1) > 0)[:, None], w, target[rows, cur].double())
    cdf = w.cumsum(-1)
    last = (cdf > u[:, :1] * cdf[:, -1:]).to(torch.int8).argmax(-1)
    path = path[:, :Nt]
    new = torch.where(path[:, 1:] >= 0, tokens.gather(1, path[:, 1:].clamp(min=0)), -1)
    new = torch.cat((new, torch.full((B, 1), -1, device=DEV)), 1)
    new[rows, count - 1] = last
    return path.int(), new.int(), count.int()


def _plain_keep(s):
    table, lens, path = s["table"].long(), s["lens"].long(), s["path"].long()
    page = s["caches"][0].shape[2]
    i = torch.arange(path.shape[1], device=DEV)[None]
    ok = i < s["count"][:, None]
    src, dst = (lens[:, None] + path)[ok], (lens[:, None] + i)[ok]
    b = torch.arange(path.shape[0], device=DEV)[:, None].expand_as(path)[ok]
    for cache in s["caches"]:
        cache[table[b, dst // page], :, dst % page] = cache[table[b, src // page], :, src % page]
    return s["lens"] + s["count"]


# -------------------------------------------------------------------- the work

def work(case):
    c = case
    if c["op"] == "verify":
        # the rows of the node where the walk ends, target's and draft's, and the walk's own numbers
        size = 4 if c["dtype"] == "float32" else 2
        rows = 1 if c["draft"] == "none" else 2
        return {"bytes": c["B"] * (rows * c["V"] * size + 20 * c["Nt"]), "flops": 3 * c["B"] * c["V"]}
    lens = _lens(c["B"], c["lo"], c["hi"])
    if c["op"] == "keep":
        # a few rows of each sequence, in every layer's keys and values: read and written
        rows = sum(min(3, c["Nt"]) for _ in lens)
        return {"bytes": rows * 2 * c["layers"] * c["Hkv"] * c["d"] * 2 * 2, "flops": 0}
    keys = sum(n + c["Nt"] for n in lens)
    rows = c["B"] * c["H"] * c["Nq"]
    return {"bytes": 4 * keys * c["Hkv"] * c["d"] + rows * (4 * c["d"] + 4) + 4 * c["B"] * c["Nt"],
            "flops": sum(4 * c["H"] * c["Nq"] * (n + (c["Nt"] + 1) // 2) * c["d"] for n in lens)}


# ----------------------------------------------------------------- the 64 bits

def exact(case, seed):
    if case["op"] != "tree":
        return None  # node numbers, tokens and copies: whole numbers, no computed values
    if case["B"] * case["H"] * case["Nq"] * case["hi"] * case["d"] > 3e11:
        return None
    return _exact_tree(prepare(case, seed))


def _exact_tree(s):
    """Row by row of the definition, one sequence and key/value head at a time; a node's ancestors
    are found by walking up from it."""
    q = s["q"].double()
    B, H, Nq, d = q.shape
    _, Hkv, page, _ = s["k_cache"].shape
    Nt = s["Nt"]
    parents = s["parents"].tolist() if s["parents"] is not None else [[j - 1 for j in range(Nt)]] * B
    o = torch.zeros((B, H, Nq, d), dtype=torch.float64, device=DEV)
    lse = torch.full((B, H, Nq), -math.inf, dtype=torch.float64, device=DEV)
    for b, n in enumerate(s["lens"].tolist()):
        nodes = sum(p >= -1 for p in parents[b])
        j = torch.arange(n + nodes, device=DEV)
        at, row = s["table"][b].long()[j // page], j % page
        hidden = torch.ones((Nq, n + nodes), dtype=torch.bool)
        for i in range(Nq):
            node = Nt - Nq + i
            if parents[b][node] < -1:
                continue
            hidden[i, :n] = False
            while node >= 0:
                hidden[i, n + node] = False
                node = parents[b][node]
        hidden = hidden.to(DEV)
        some = ~hidden.all(-1)
        for h in range(Hkv):
            heads = slice(h * (H // Hkv), (h + 1) * (H // Hkv))
            k, v = (s[x][at, h, row].double() for x in ("k_cache", "v_cache"))
            x = (q[b, heads] @ k.T / math.sqrt(d)).masked_fill(hidden, -math.inf)
            o[b, heads] = torch.where(some[None, :, None], torch.softmax(x, -1) @ v, 0.0)
            lse[b, heads] = torch.logsumexp(x, -1)
    return o, lse
