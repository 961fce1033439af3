"""Float64 oracle of speculative decoding over a paged bf16 cache: attention of drafted trees,
their verification, and the rows that are kept.  Loops over the definitions, on the CPU."""
from __future__ import annotations

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
