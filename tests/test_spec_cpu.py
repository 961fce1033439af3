"""Speculative decoding without a GPU: its oracle's pins, and every refusal of the entry points
(all of which return before anything touches CUDA)."""
import ctypes
import itertools
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import spec
from test_boundary_cpu import fa  # noqa: F401

P = 0x10000  # aligned, never dereferenced


# ------------------------------------------------------------------------ pins

def test_ancestors():
    parents = [-1, 0, 0, 1, 3, -2, 2]
    assert spec.ancestors(parents, 4) == [4, 3, 1, 0] and spec.ancestors(parents, 6) == [6, 2, 0]
    assert spec.ancestors(parents, 5) == [] and spec.ancestors([-1, -1], 1) == [1]


def test_tree_attention_is_attention_over_the_path():
    """Each row is plain softmax attention over the contiguous keys of its own path."""
    rng = np.random.default_rng(0)
    kc, vc = rng.standard_normal((2, 7, 1, 4, 8))
    q = rng.standard_normal((1, 2, 3, 8))
    table, n = np.array([[4, 1, 6]]), 5
    parents = np.array([[-1, 0, 0, 2]])
    o, lse, _ = spec.decode_tree(q, kc, vc, table, [n], parents, 0.5)
    k, v = (np.concatenate([c[p, 0] for p in (4, 1, 6)]) for c in (kc, vc))
    for i, path in enumerate(([0, 1], [0, 2], [0, 2, 3])):
        keys = list(range(n)) + [n + j for j in path]
        for h in range(2):
            s = 0.5 * (k[keys] @ q[0, h, i])
            p = np.exp(s)
            assert np.allclose(o[0, h, i], p @ v[keys] / p.sum(), atol=1e-13)
            assert np.isclose(lse[0, h, i], np.log(p.sum()))
    chain, _, _ = spec.decode_tree(q, kc, vc, table, [n], None, 0.5)
    assert np.allclose(chain, spec.decode_tree(q, kc, vc, table, [n], np.array([[-1, 0, 1]]), 0.5)[0])
    none, l, _ = spec.decode_tree(q, kc, vc, table, [n], np.array([[-1, -2, 0]]), 0.5)
    assert np.all(none[:, :, 1] == 0) and np.all(np.isneginf(l[:, :, 1])) and np.isfinite(l[:, :, 2]).all()


def _first_token_distribution(p, q, drafts, weight, certain=False, replacement=True):
    """The distribution of the first new token over all of `drafts` (tuples of tokens tried under the
    root, of probability `weight`) and over uniforms on a grid of cells, in exact fractions: the
    acceptance of a child is a threshold on its own uniform, so the oracle's decisions are counted
    at the middle of 1/N cells and the thresholds are exact where N is a multiple of the
    denominators."""
    V = len(p)
    total = [Fraction(0)] * V
    for d in drafts:
        Nt = 1 + len(d)
        target = np.array([[float(x) for x in p]] * Nt)
        draft = None if certain else np.array([[float(x) for x in q]] * Nt)
        parents = [-1] + [0] * len(d)
        alive = Fraction(1)  # probability that the children so far were rejected
        for k, x in enumerate(d):
            # the threshold of child k, given that the ones before it were rejected (u = 1 - eps)
            N = 1 << 12
            u = np.full(Nt, 1 - 2.0 ** -24)

            def accepted(cell):
                u[k + 1] = (cell + 0.5) / N
                path, _ = spec.verify([0, *d], parents, target, draft, u, replacement)
                return len(path) > 1 and path[1] == k + 1
            lo, hi = 0, N  # accepted for cells below the threshold
            while lo < hi:
                mid = (lo + hi) // 2
                lo, hi = (mid + 1, hi) if accepted(mid) else (lo, mid)
            total[x] += weight(d) * alive * Fraction(lo, N)
            alive *= 1 - Fraction(lo, N)
        # behind the last rejection: the last token's distribution, from the thresholds of u[0]
        u = np.full(Nt, 1 - 2.0 ** -24)
        counts = [0] * V
        N = 1 << 10
        for cell in range(N):
            u[0] = (cell + 0.5) / N
            path, new = spec.verify([0, *d], parents, target, draft, u, replacement)
            if len(path) == 1:
                counts[new[0]] += 1
        for i in range(V):
            total[i] += weight(d) * alive * Fraction(counts[i], N)
    return [float(x) for x in total]


P3, Q3 = [Fraction(1, 2), Fraction(3, 8), Fraction(1, 8)], [Fraction(1, 4), Fraction(1, 4), Fraction(1, 2)]


def test_verification_keeps_the_targets_distribution():
    """Summed over all drafts, the first new token is distributed as the target says (the grids are
    good to 2^-10 per threshold)."""
    def independent(d):
        return Fraction(np.prod([float(Q3[x]) for x in d]))

    def without(d):
        w, left = Fraction(1), Fraction(1)
        for x in d:
            w *= Q3[x] / left
            left -= Q3[x]
        return w
    for n in (1, 2):
        got = _first_token_distribution(P3, Q3, list(itertools.product(range(3), repeat=n)), independent)
        assert np.allclose(got, [float(x) for x in P3], atol=n * 2.0 ** -9), got
    got = _first_token_distribution(P3, Q3, list(itertools.permutations(range(3), 2)), without, replacement=False)
    assert np.allclose(got, [float(x) for x in P3], atol=2.0 ** -8), got
    for d in [(0,), (2, 1), (1, 1)]:
        got = _first_token_distribution(P3, Q3, [d], lambda _: Fraction(1), certain=True)
        assert np.allclose(got, [float(x) for x in P3], atol=2.0 ** -8), got


def test_verification_of_a_chain():
    target = np.eye(4)[[1, 2, 3]]
    draft = np.eye(4)[[1, 2, 0]]
    assert spec.verify([0, 1, 2], None, target, draft, [0.5] * 3) == ([0, 1, 2], [1, 2, 3])
    assert spec.verify([0, 1, 0], None, target, np.eye(4)[[1, 0, 0]], [0.5] * 3) == ([0, 1], [1, 2])
    assert spec.verify([0, 1, 2], [-2, -2, -2], target, draft, [0.5] * 3) == ([], [])


def test_keep_moves_rows_as_if_at_once():
    cache = np.arange(6 * 1 * 2 * 1, dtype=float).reshape(6, 1, 2, 1)
    table = np.array([[3, 0, 5]])
    new = spec.keep(cache, table, [1], np.array([[1, 2, 4]]), [3])
    rows = [new[p, 0, r, 0] for p in (3, 0, 5) for r in range(2)]
    old = [cache[p, 0, r, 0] for p in (3, 0, 5) for r in range(2)]
    assert rows == [old[0], old[2], old[3], old[5], old[4], old[5]]


# -------------------------------------------------------------------- refusals

TREE = dict(q=P, k_cache=P, v_cache=P, block_table=P, seq_lens=P, parents=P, o=P, lse=P, B=2, H=4, Hkv=2,
            Nq=3, Nt=5, d=128, ps=16, mp=4, num=9, scale=0.1, ws=None, ws_bytes=0, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), 1), (dict(k_cache=None), 1), (dict(v_cache=None), 1), (dict(block_table=None), 1),
    (dict(seq_lens=None), 1), (dict(o=None), 1), (dict(lse=None), 1), (dict(B=0), 1), (dict(H=3), 1),
    (dict(Hkv=8), 1), (dict(Nq=0), 1), (dict(Nq=6), 1), (dict(Nt=2), 1), (dict(Nt=257), 2), (dict(ps=0), 1),
    (dict(mp=0), 1), (dict(num=0), 1), (dict(num=1 << 30), 1), (dict(ps=1 << 20, mp=1 << 11), 1),
    (dict(ps=1 << 10, mp=(1 << 21) - 1), 1), (dict(B=1 << 20, mp=1 << 11), 1), (dict(B=1 << 23, Nt=256), 1),
    (dict(d=80), 2), (dict(d=192), 2), (dict(scale=0.0), 1), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(q=P + 8), 3), (dict(k_cache=P + 2), 3), (dict(v_cache=P + 8), 3),
    (dict(o=P + 8), 3), (dict(lse=P + 2), 3), (dict(parents=P + 1), 3), (dict(block_table=P + 2), 3),
    (dict(seq_lens=P + 2), 3), (dict(ws=P + 8), 3), (dict(), 6), (dict(parents=None), 6),
])
def test_tree_rejects_bad_arguments(fa, kw, code):  # noqa: F811
    assert fa.fa_decode_paged_tree(*{**TREE, **kw}.values()) == code


def test_tree_workspace_of_invalid_sizes(fa):  # noqa: F811
    assert fa.fa_decode_paged_tree_workspace_bytes(1, 4, 3, 1, 1, 128, 16, 4) == 0
    assert fa.fa_decode_paged_tree_workspace_bytes(1, 4, 4, 1, 1, 80, 16, 4) == 0
    assert fa.fa_decode_paged_tree_workspace_bytes(1, 4, 4, 2, 1, 128, 16, 4) == 0
    assert fa.fa_decode_paged_tree_workspace_bytes(1, 4, 4, 1, 257, 128, 16, 4) == 0


VERIFY = dict(tokens=P, parents=P, target=P, draft=P, uniform=P, path=P, new=P, count=P, B=2, Nt=5, V=100,
              bf16=0, replacement=1, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=None), 1), (dict(target=None), 1), (dict(uniform=None), 1), (dict(path=None), 1),
    (dict(new=None), 1), (dict(count=None), 1), (dict(B=0), 1), (dict(Nt=0), 1), (dict(V=0), 1),
    (dict(V=(1 << 30) + 1), 1), (dict(B=1 << 26), 1), (dict(Nt=257), 2), (dict(target=P + 8), 3),
    (dict(draft=P + 8), 3), (dict(tokens=P + 2), 3), (dict(parents=P + 1), 3), (dict(uniform=P + 2), 3),
    (dict(path=P + 2), 3), (dict(new=P + 2), 3), (dict(count=P + 2), 3),
])
def test_verify_rejects_bad_arguments(fa, kw, code):  # noqa: F811
    assert fa.fa_verify_tree(*{**VERIFY, **kw}.values()) == code


KEEP = dict(caches=(P,), n=1, block_table=P, seq_lens=P, path=P, count=P, lens=P, B=2, Nt=5, Hkv=2, d=128, ps=16,
            mp=4, num=9, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(caches=None), 1), (dict(caches=(0,)), 1), (dict(n=0), 1), (dict(n=129), 1), (dict(block_table=None), 1),
    (dict(seq_lens=None), 1), (dict(path=None), 1), (dict(count=None), 1), (dict(lens=None), 1), (dict(B=0), 1),
    (dict(B=65536), 1), (dict(Nt=0), 1), (dict(Hkv=0), 1), (dict(ps=0), 1), (dict(mp=0), 1), (dict(num=0), 1),
    (dict(ps=1 << 20, mp=1 << 11), 1), (dict(num=1 << 30), 1), (dict(Nt=257), 2), (dict(d=80), 2), (dict(d=0), 2),
    (dict(caches=(P + 8,)), 3), (dict(block_table=P + 2), 3), (dict(seq_lens=P + 2), 3), (dict(path=P + 2), 3),
    (dict(count=P + 2), 3), (dict(lens=P + 2), 3), (dict(caches=(P, 2 * P, P), n=3), 1),
])
def test_keep_rejects_bad_arguments(fa, kw, code):  # noqa: F811
    a = {**KEEP, **kw}
    if a["caches"] is not None:
        a["caches"] = (ctypes.c_void_p * len(a["caches"]))(*a["caches"])
    assert fa.fa_keep_path(*a.values()) == code


def _cpu():
    k = torch.zeros((4, 2, 8, 64), dtype=torch.bfloat16)
    i = torch.zeros((2, 3), dtype=torch.int32)
    return k, i, torch.zeros((2, 4, 3, 64), dtype=torch.bfloat16)


def test_wrappers_reject_cpu_tensors(fa):  # noqa: F811
    k, i, q = _cpu()
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        fa.decode_paged_tree(q, k, k, i, i[:, 0], i)
    with pytest.raises(ValueError, match="tokens must be a CUDA tensor"):
        fa.verify_tree(i, i, torch.zeros(2, 3, 5), None, torch.zeros(2, 3))
    with pytest.raises(ValueError, match="block_table must be a CUDA tensor"):
        fa.keep_path([k], i, i[:, 0], i, i[:, 0])
    with pytest.raises(ValueError, match="1 to 128"):
        fa.keep_path([], i, i[:, 0], i, i[:, 0])
