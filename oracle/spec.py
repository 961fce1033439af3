"""Float64 oracle of speculative decoding over a paged bf16 cache: attention of drafted trees,
their verification, and the rows that are kept.  Loops over the definitions, on the CPU."""
from __future__ import annotations

from fractions import Fraction

import numpy as np


def parents_of(parents, Nt):
    """The parents of one tree as a list (None: a chain)."""
    return [j - 1 for j in range(Nt)] if parents is None else [int(p) for p in parents]


def ancestors(parents, j):
    """Node j and those above it; empty where there is no node."""
    if parents[j] < -1:
        return []
    found = []
    while j >= 0:
        found.append(j)
        j = parents[j]
    return found


def decode_tree(q, kc, vc, table, lens, parents, scale):
    """q [B,H,Nq,d], caches [pages,Hkv,page,d] in float64, table [B,width], lens [B], parents [B,Nt]
    or None.  Returns (o, lse, (pv, qk)): the outputs and, for error bounds, per element the sum of
    |p v| and per row the largest sum of |q k| scale of the keys it sees."""
    B, H, Nq, d = q.shape
    _, Hkv, page, _ = kc.shape
    G = H // Hkv
    o, pv = np.zeros(q.shape), np.zeros(q.shape)
    lse, qk = np.full((B, H, Nq), -np.inf), np.zeros((B, H, Nq))
    for b in range(B):
        Nt = Nq if parents is None else parents.shape[1]
        par = parents_of(None if parents is None else parents[b], Nt)
        n = int(lens[b])
        for i in range(Nq):
            nodes = ancestors(par, Nt - Nq + i)
            if not nodes:
                continue
            keys = np.concatenate([np.arange(n), n + np.array(sorted(nodes))])
            at, row = table[b][keys // page], keys % page
            for kvh in range(Hkv):
                k, v = kc[at, kvh, row], vc[at, kvh, row]
                for h in range(kvh * G, kvh * G + G):
                    with np.errstate(invalid="ignore", over="ignore"):
                        s = scale * (k @ q[b, h, i])
                        m = s.max()
                        p = np.exp(s - (m if m > -np.inf else 0.0))
                        total = p.sum()
                        if total == 0:
                            continue
                        p /= total
                        o[b, h, i] = p @ v
                        pv[b, h, i] = p @ np.abs(v)
                        lse[b, h, i] = m + np.log(total)
                        qk[b, h, i] = scale * (np.abs(k) @ np.abs(q[b, h, i])).max()
    return o, lse, (pv, qk)


def verify(tokens, parents, target, draft, uniform, replacement=True):
    """One sequence, in exact fractions: tokens, parents (None: a chain), uniform [Nt]; target, draft
    (or None) [Nt, V].  Returns (path, new_tokens)."""
    Nt, V = target.shape
    par = parents_of(parents, Nt)
    if par[0] < -1:
        return [], []

    def row(x):
        return [Fraction(float(v)) for v in x]

    cur, path, new = 0, [0], []
    while True:
        p = row(target[cur])
        q = None if draft is None else row(draft[cur])
        a, used, total, gone = Fraction(0), Fraction(0), Fraction(1), set()
        accepted = None
        for j in range(cur + 1, Nt):
            if par[j] != cur:
                continue
            x, u = int(tokens[j]), Fraction(float(uniform[j]))
            if q is None:
                w = Fraction(0) if x in gone else p[x]
                if u * total < w:
                    accepted = j
                    break
                gone.add(x)
                total -= w
            else:
                rest = Fraction(1) if replacement else max(1 - used, Fraction(1, 2 ** 60))
                if u * q[x] / rest * total < max(p[x] - a * q[x], 0):
                    accepted = j
                    break
                a = min(a + total / rest, Fraction(2 ** 60))
                used += q[x]
                total = sum(max(pi - a * qi, 0) for pi, qi in zip(p, q))
        if accepted is None:
            break
        cur = accepted
        path.append(cur)
        new.append(int(tokens[cur]))
    left = [0 if i in gone else p[i] for i in range(V)] if q is None else [max(pi - a * qi, 0) for pi, qi in zip(p, q)]
    if sum(left) == 0:
        left = p
    goal, run = Fraction(float(uniform[0])) * sum(left), Fraction(0)
    for i in range(V):
        run += left[i]
        if run > goal:
            return path, new + [i]
    return path, new + [-1]


def keep(cache, table, lens, path, count):
    """cache [pages, Hkv, page, d] with the rows of the accepted nodes in their new places."""
    old, new = cache, cache.copy()
    page = cache.shape[2]
    for b in range(len(lens)):
        for i in range(int(count[b])):
            src, dst = int(lens[b]) + int(path[b, i]), int(lens[b]) + i
            new[table[b, dst // page], :, dst % page] = old[table[b, src // page], :, src % page]
    return new
