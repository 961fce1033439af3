"""Helpers of the paged e4m3 cache tests: seeded caches and the bounds of the decode."""
from __future__ import annotations

import numpy as np
import torch

from oracle import cache as oc

DEV = "cuda:0"


def make_cache(num_pages, Hkv, ps, d, group, seed, spread=1.0, pow2=False):
    """Random codes (no NaN) and scales of one cache, on the CPU."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((num_pages, Hkv, ps // group, group * d), generator=g)
    x = x * torch.exp(spread * torch.randn((num_pages, Hkv, ps // group, 1), generator=g))
    scale = x.abs().amax(-1, keepdim=True) / 448
    if pow2:
        scale = torch.exp2(torch.ceil(torch.log2(scale)))
    codes = (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes.reshape(num_pages, Hkv, ps, d).contiguous(), scale.squeeze(-1).contiguous()


def make_table(lens, ps, width, num_pages, seed, unused=-1):
    """Table rows of distinct random pages; entries behind the last page are `unused`."""
    g = torch.Generator().manual_seed(seed)
    perm = torch.randperm(num_pages, generator=g).to(torch.int32)
    table = torch.full((len(lens), width), unused, dtype=torch.int32)
    at = 0
    for b, n in enumerate(lens):
        need = -(-int(n) // ps)
        table[b, :need] = perm[at:at + need]
        at += need
    assert at <= num_pages
    return table


def check_decode(o, lse, ref, what=""):
    """o (bf16 values) and lse against the oracle's (o, lse, terms), element by element.

    The bound, from where the operation may round (u32 = 2^-24; half a bf16 step is 2^-8 of the
    value): a score is a sum of d products in fp32, whose error is allowed 16 u32 of the sum of
    its magnitudes (2^-20), and shifts L by at most that and every p by twice that relatively; p
    times its value scale is rounded to f16's 11 bits (2^-11 relative, or half of its smallest
    step, 2^-25) and kept as three e5m2 numbers of 3 bits, the first two truncated, which leaves
    less than 2^-5 of the value, or e5m2's smallest step 2^-16; the third, of 2^5 times that, is
    rounded to half a step of 3 bits: 2^-9 relative, or 2^-20.  Here 2^9 stands for a reference
    that is at most the row's largest p times 16 times the head's largest value scale, so the
    absolute error of p times the scale is at most (2^-20 + 2^-25) 2^-9 2^4 < 2^-24 of those two's
    product, and it meets each code once; the sums over keys and L itself are fp32 (2^-16
    relative for up to 2^8 accumulation steps of u32); O is rounded to bf16."""
    ro, rl, (pv, vmax, qk) = ref
    o, lse = np.asarray(o, dtype=np.float64), np.asarray(lse, dtype=np.float64)
    es = 2.0 ** -20 * qk
    empty = ~np.isfinite(rl)
    assert np.array_equal(np.isneginf(lse), empty), f"{what}: rows without keys"
    assert np.all(o[empty] == 0), f"{what}: O of rows without keys"
    bl = es + 2.0 ** -20 * (1 + np.abs(np.where(empty, 0, rl)))
    el = np.where(empty, 0, np.abs(np.where(empty, 0, lse) - np.where(empty, 0, rl)))
    assert np.all(el <= bl), f"{what}: L off by {el.max():.3e}, worst ratio {(el / bl).max():.2f}"
    bo = (2.0 ** -8 * np.abs(ro) + (2.0 ** -9 + 2.0 ** -11 + 2.0 ** -16 + 2 * es[..., None]) * pv * (1 + 2.0 ** -8)
          + 2.0 ** -24 * vmax + 1e-30)
    eo = np.abs(o - ro)
    assert np.all(eo <= bo), f"{what}: O off by {eo.max():.3e}, worst ratio {(eo / bo).max():.2f}"
    return float((eo / bo).max()), float((el / bl).max())


def oracle_decode(q, kc, vc, ks, vs, table, lens, causal, scale):
    n = [t.detach().cpu().numpy() for t in (kc, vc, ks, vs, table, lens)]
    return oc.decode(q.detach().cpu().double().numpy(), *n, causal, scale)
