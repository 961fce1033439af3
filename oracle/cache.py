"""The paged e4m3 key/value cache on the CPU: storing, attention, page bookkeeping.

TEST INFRASTRUCTURE ONLY, like the rest of this package: the definitions written out in
numpy float64 and Python integers, one token, row or page at a time, sharing no code with
the CUDA library.
"""
from __future__ import annotations

import numpy as np

from .fp8 import e4m3_round, e4m3_value

NAN_CODE = 0x7F


def least_scale(amax: float) -> float:
    """The smallest power of two s >= 2^-126 with amax <= 448 s."""
    s = 2.0 ** -126
    while amax > 448.0 * s:
        s *= 2.0
    return s


def pow2_at_least(x: float) -> float:
    """The smallest power of two >= x (0 for 0)."""
    return 0.0 if x == 0 else float(2.0 ** np.ceil(np.log2(x)))


def encode(x) -> np.ndarray:
    """e4m3 codes of x: nearest even; NaN and infinities become the NaN code."""
    x = np.asarray(x, dtype=np.float64)
    fin = np.isfinite(x)
    return np.where(fin, e4m3_round(np.where(fin, x, 0.0)), NAN_CODE).astype(np.uint8)


def append(x, codes, scale, table, lens, cu):
    """Store x [T, Hkv, d] (float64) in copies of codes [pages, Hkv, ps, d] and scale
    [pages, Hkv, groups]; returns the copies (scales as float32, exactly)."""
    codes, scale = codes.copy(), scale.copy()
    size = codes.shape[2] // scale.shape[2]
    ps = codes.shape[2]
    for b in range(len(lens)):
        start, n = int(lens[b]), int(cu[b + 1] - cu[b])
        j = start
        while j < start + n:
            stop = min(start + n, (j // size + 1) * size)
            page, g = int(table[b, j // ps]), j % ps // size
            for h in range(codes.shape[1]):
                new = x[cu[b] + j - start:cu[b] + stop - start, h]
                fin = np.abs(new[np.isfinite(new)])
                s = least_scale(float(fin.max()) if fin.size else 0.0)
                if j % size:
                    old = float(scale[page, h, g])
                    s = max(s, pow2_at_least(old))
                    if s > old:
                        r = slice(g * size, j % ps)
                        codes[page, h, r] = encode(e4m3_value(codes[page, h, r]) * (old / s))
                scale[page, h, g] = s
                codes[page, h, j % ps:j % ps + stop - j] = encode(new / s)
            j = stop
    return codes, scale


def gather(codes, scale, table_row, n, h):
    """float64 [n, d]: the first n cached tokens of one sequence and head."""
    ps = codes.shape[2]
    size = ps // scale.shape[2]
    j = np.arange(n)
    page, row = np.asarray(table_row, dtype=np.int64)[j // ps], j % ps
    return e4m3_value(codes[page, h, row]) * scale[page, h, row // size].astype(np.float64)[:, None]


def decode(q, k_codes, v_codes, k_scale, v_scale, table, lens, causal, scale):
    """(o, lse, terms): float64 attention of q [B, H, Nq, d]; terms holds per row what error
    bounds need: sum_j p_j |v_j| per column, sum_j |code of v_j| times p_max and the largest value
    scale of the head's n tokens, and the largest over the seen keys of scale * sum_c |q_c k_c|."""
    B, H, Nq, d = q.shape
    Hkv = k_codes.shape[1]
    o = np.zeros((B, H, Nq, d))
    lse = np.full((B, H, Nq), -np.inf)
    pv, vmax, qk = np.zeros((B, H, Nq, d)), np.zeros((B, H, Nq, d)), np.zeros((B, H, Nq))
    for b in range(B):
        n = int(lens[b])
        for h in range(H):
            kvh = h // (H // Hkv)
            k = gather(k_codes, k_scale, table[b], n, kvh)
            v = gather(v_codes, v_scale, table[b], n, kvh)
            codes = np.abs(gather(v_codes, np.ones_like(v_scale), table[b], n, kvh))
            ps, groups = v_codes.shape[2], v_scale.shape[2]
            at = np.arange(n)
            largest = v_scale[table[b][at // ps], kvh, at % ps // (ps // groups)].max(initial=0.0)
            for i in range(Nq):
                end = max(0, min(n, n - Nq + 1 + i)) if causal else n
                if end == 0:
                    continue
                s = scale * (k[:end] @ q[b, h, i])
                m = s.max()
                p = np.exp(s - m)
                lse[b, h, i] = m + np.log(p.sum())
                p /= p.sum()
                o[b, h, i] = p @ v[:end]
                pv[b, h, i] = p @ np.abs(v[:end])
                vmax[b, h, i] = p.max() * float(largest) * codes[:end].sum(0)
                qk[b, h, i] = scale * (np.abs(k[:end]) @ np.abs(q[b, h, i])).max()
    return o, lse, (pv, vmax, qk)


def _need(n, ps, width):
    return min(max(0, -(-int(n) // ps)), width)


def live_pages(table, lens, ps, num_pages):
    used = set()
    for b in range(len(lens)):
        for c in range(_need(lens[b], ps, table.shape[1])):
            if 0 <= table[b, c] < num_pages:
                used.add(int(table[b, c]))
    return used


def free(table, lens, ps, num_pages):
    used = live_pages(table, lens, ps, num_pages)
    pages = [p for p in range(num_pages) if p not in used]
    return pages + [-1] * (num_pages - len(pages)), len(pages)


def fork(table, lens, parents, fresh, ps):
    n, width = len(parents), table.shape[1]
    rows = np.full((n, width), -1)
    out = np.zeros(n, dtype=int)
    src, dst = np.full(n, -1), np.full(n, -1)
    for i, parent in enumerate(parents):
        out[i] = lens[parent]
        need = _need(lens[parent], ps, width)
        rows[i, :need] = table[parent, :need]
        if lens[parent] % ps:
            src[i], dst[i] = table[parent, need - 1], fresh[i]
            rows[i, need - 1] = fresh[i]
    return rows, out, src, dst


def compact(table, lens, ps, num_pages):
    used = live_pages(table, lens, ps, num_pages)
    n = len(used)
    src = sorted(p for p in used if p >= n)
    dst = [p for p in range(n) if p not in used]
    to = dict(zip(src, dst))
    new = table.copy()
    for b in range(len(lens)):
        for c in range(_need(lens[b], ps, table.shape[1])):
            new[b, c] = to.get(int(table[b, c]), table[b, c])
    pad = [-1] * (max(1, num_pages // 2) - len(src))
    return new, src + pad, dst + pad, n, len(src)
