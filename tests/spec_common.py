"""Helpers of the speculative decoding tests: seeded caches and trees, and the bounds."""
from __future__ import annotations

import numpy as np
import torch

from oracle import spec

DEV = "cuda:0"


def random_trees(B, Nt, seed, ragged=False, bushy=True):
    """parents int32 [B, Nt] of random trees under node 0; ragged: with missing nodes at the end."""
    g = np.random.default_rng(seed)
    out = np.full((B, Nt), -2, dtype=np.int32)
    for b in range(B):
        n = int(g.integers(0, Nt + 1)) if ragged else Nt
        for j in range(n):
            u = g.random()
            out[b, j] = -1 if j == 0 else min(j - 1, int((u * u if bushy else np.sqrt(u)) * j))
    return torch.from_numpy(out)


def make_paged(lens, Nt, page, Hkv, d, seed, spare=3, width=None, fill=None):
    """A bf16 cache with scattered pages for lens[b] + Nt tokens each: k, v, table (CPU; entries
    behind the last page are -1).  `fill`: the value of every place without a token."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-(n + Nt) // page) for n in lens]
    pages = sum(need) + spare
    k, v = (torch.randn((pages, Hkv, page, d), generator=g).bfloat16() for _ in "kv")
    perm = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((len(lens), width or max(need)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    if fill is not None:
        used = torch.zeros((pages, page), dtype=torch.bool)
        for b, n in enumerate(lens):
            j = torch.arange(n + Nt)
            used[table[b].long()[j // page], j % page] = True
        empty = ~used[:, None, :, None].expand_as(k)
        k[empty], v[empty] = fill, fill
    return k, v, table


def oracle_tree(q, k, v, table, lens, parents, scale=None):
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    n = [t.detach().cpu().double().numpy() for t in (q, k, v)]
    return spec.decode_tree(*n, table.cpu().numpy(), [int(x) for x in lens],
                            None if parents is None else parents.cpu().numpy(), scale)


def check_tree(o, lse, ref, what=""):
    """o and lse against the oracle's, element by element.

    A score is a sum of d exact products in fp32, each step off by at most 2^-23 of the sum of
    magnitudes (the tensor cores may truncate): es = d 2^-23 qk, which shifts L by at most es and
    every p by 2 es relatively.  P is rounded to bf16, 2^-8 of each term; sums over keys are fp32
    (2^-16 relative for up to 2^8 steps); L is fp32, its logarithm and exponentials good to
    2^-20; O is rounded to bf16, 2^-8 of the value."""
    ro, rl, (pv, qk) = ref
    o, lse = (t.detach().cpu().double().numpy() for t in (o, lse))
    es = o.shape[-1] * 2.0 ** -23 * qk
    none = np.isneginf(rl)
    assert np.array_equal(np.isneginf(lse), none), f"{what}: rows without keys"
    assert np.all(o[none] == 0), f"{what}: O of rows without keys"
    assert np.array_equal(np.isnan(lse), np.isnan(rl)), f"{what}: NaN in L"
    some = np.isfinite(rl)
    bl = (es + 2.0 ** -20 * (1 + np.abs(rl)))[some]
    el = np.abs(lse[some] - rl[some])
    assert np.all(el <= bl), f"{what}: L off by {el.max():.3e}, worst ratio {(el / bl).max():.2f}"
    assert np.array_equal(np.isnan(o), np.isnan(ro)), f"{what}: NaN in O"
    inf = np.isinf(ro)
    assert np.array_equal(o[inf], ro[inf]) and np.all(np.isinf(o) == inf), f"{what}: infinities in O"
    fin = np.isfinite(ro)
    bo = 2.0 ** -8 * np.abs(np.where(fin, ro, 0)) + (2.0 ** -8 + 2.0 ** -16 + 2 * es[..., None]) * pv * (1 + 2.0 ** -8) + 1e-30
    eo, bo = np.abs(o[fin] - ro[fin]), bo[fin]
    assert np.all(eo <= bo), f"{what}: O off by {eo.max():.3e}, worst ratio {(eo / bo).max():.2f}"
