"""Attention of drafted trees whose rows fill a part of a block only, so that some warps have few rows
or none, against the float64 oracle."""
from __future__ import annotations

import pytest
import torch

from gpu_common import load_fa
from spec_common import DEV, check_tree, make_paged, oracle_tree, random_trees

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    return load_fa()


def inputs(lens, G, Hkv, Nt, Nq, d, page, seed, par):
    k, v, table = make_paged(lens, Nt, page, Hkv, d, seed)
    q = torch.randn((len(lens), G * Hkv, Nq, d), generator=torch.Generator().manual_seed(seed + 1)).bfloat16()
    return q, k, v, table, torch.tensor(lens, dtype=torch.int32), par


def check(fa, args):
    q, k, v, table, lens, par = args
    dev = [None if t is None else t.to(DEV) for t in args]
    o, lse = fa.decode_paged_tree(*dev)
    assert fa.fa_device_status() == fa.FA_OK
    check_tree(o, lse, oracle_tree(q, k, v, table, lens, par))
    for _ in range(5):
        o2, lse2 = fa.decode_paged_tree(*dev)
        assert torch.equal(o.view(torch.int16), o2.view(torch.int16)) and torch.equal(lse, lse2)


@pytest.mark.parametrize("G,Nt", [(1, 1), (1, 31), (4, 8), (1, 33), (8, 6), (3, 21), (16, 4), (1, 65), (9, 7)])
@pytest.mark.parametrize("d", [64, 96])
def test_rows(fa, d, G, Nt):
    """From one row to just above 64, in trees with missing nodes, of one and of several tiles."""
    lens = [0, 127, 1500, 40, 777]
    check(fa, inputs(lens, G, 2, Nt, Nt, d, 16, G + Nt, random_trees(len(lens), Nt, Nt, ragged=True)))


@pytest.mark.parametrize("G,Nq", [(8, 4), (16, 3), (2, 1)])
def test_long_chain(fa, G, Nq):
    check(fa, inputs([20001, 3, 6000], G, 1, Nq, Nq, 64, 32, Nq, None))


@pytest.mark.parametrize("G", [3, 6])
def test_large_scores(fa, G):
    """Scores that grow along the keys, so that the reference of the exponents moves again and again."""
    lens, Nt = [1000, 640], 10
    q, k, v, table, n, par = inputs(lens, G, 2, Nt, Nt, 64, 16, 5, random_trees(2, Nt, 6))
    q[..., 0] = 8.0
    for b, length in enumerate(lens):
        for key in range(length + Nt):
            k[table[b, key // 16], :, key % 16, 0] = key / 16.0
    check(fa, (q, k, v, table, n, par))


@pytest.mark.parametrize("G", [2, 5])
@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
def test_values_that_are_not_finite(fa, value, G):
    """Of cached tokens, which all rows see, and of a node, which some do."""
    lens, Nt, page = [300, 126], 11, 16
    q, k, v, table, n, par = inputs(lens, G, 1, Nt, Nt, 64, page, 9, random_trees(2, Nt, 10))
    for b, length in enumerate(lens):
        for key, c in ((7, 3), (length - 1, 40), (length + 2, 63), (length + 6, 5)):
            v[table[b, key // page], :, key % page, c] = value
    check(fa, (q, k, v, table, n, par))


@pytest.mark.parametrize("Nt", [32, 33, 200, 256])
@pytest.mark.parametrize("d", [64, 128])
def test_deep_trees(fa, d, Nt):
    """A path as long as the tree, a comb of it (each second node a leaf), and one that ends early; the
    path is what no parents at all stand for."""
    j = torch.arange(Nt)
    comb = torch.where(j % 2 == 1, j - 1, j - 2).clamp(min=-1)
    short = torch.where(j < Nt - 7, j - 1, -2)
    par = torch.stack([j - 1, comb, short]).to(torch.int32)
    args = inputs([130, 5, 0], 1, 2, Nt, Nt, d, 16, Nt, par)
    check(fa, args)
    dev = [t.to(DEV) for t in args]
    o, lse = fa.decode_paged_tree(*dev)
    o2, lse2 = fa.decode_paged_tree(*dev[:5])
    assert torch.equal(o[0], o2[0]) and torch.equal(lse[0], lse2[0])
