"""Attention of drafted trees over a paged bf16 cache against the float64 oracle."""
from __future__ import annotations

import pytest
import torch

from gpu_common import load_fa
from spec_common import DEV, check_tree, make_paged, oracle_tree, random_trees

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    return load_fa()


def run(fa, lens, H, Hkv, Nt, Nq, d, page, seed, parents="random", fill=None, scale=None, what=""):
    B = len(lens)
    k, v, table = make_paged(lens, Nt, page, Hkv, d, seed, fill=fill)
    g = torch.Generator().manual_seed(seed + 1)
    q = torch.randn((B, H, Nq, d), generator=g).bfloat16()
    par = random_trees(B, Nt, seed + 2, ragged=parents == "ragged") if isinstance(parents, str) else parents
    dev = [t.to(DEV) if t is not None else None
           for t in (q, k, v, table, torch.tensor(lens, dtype=torch.int32), par)]
    o, lse = fa.decode_paged_tree(*dev, scale=scale)
    assert fa.fa_device_status() == fa.FA_OK
    check_tree(o, lse, oracle_tree(q, k, v, table, lens, par, scale), what)
    return dev, (o, lse)


@pytest.mark.parametrize("d", [64, 96, 128, 256])
@pytest.mark.parametrize("H,Hkv,Nt,Nq", [(4, 2, 7, 7), (8, 1, 33, 33), (6, 2, 20, 9), (1, 1, 1, 1)])
def test_sizes(fa, d, H, Hkv, Nt, Nq):
    run(fa, [0, 1, 100, 127, 128, 129, 300], H, Hkv, Nt, Nq, d, 16, d + Nt)


@pytest.mark.parametrize("page", [1, 2, 5, 8, 24, 48, 100, 256])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_pages(fa, page, d):
    run(fa, [3, 250, 64], 4, 2, 12, 12, d, page, page)


@pytest.mark.parametrize("H,Hkv,Nt,d", [(16, 1, 8, 128), (12, 1, 11, 64), (24, 2, 32, 128), (8, 1, 48, 96),
                                        (16, 2, 21, 256), (4, 1, 130, 128), (2, 1, 256, 64), (3, 1, 200, 128)])
def test_many_rows(fa, H, Hkv, Nt, d):
    """One and two blocks of 128 rows, items of both in one call, and trees wider than a tile."""
    run(fa, [77, 5, 400], H, Hkv, Nt, Nt, d, 32, Nt, parents="ragged")


@pytest.mark.parametrize("H,Hkv,Nt,d", [(16, 2, 21, 256), (48, 4, 32, 128), (16, 2, 21, 64)])
def test_many_rows_of_several_tiles(fa, H, Hkv, Nt, d):
    """Items of different numbers of rows in turn, each of several tiles, in calls right after one another."""
    dev, (o, lse) = run(fa, [1830, 761, 249, 1422, 353], H, Hkv, Nt, Nt, d, 48, Nt, parents="ragged")
    for _ in range(20):
        o2, lse2 = fa.decode_paged_tree(*dev)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("Nq", [1, 4, 19])
def test_chain(fa, Nq):
    run(fa, [0, 1, 60, 500], 8, 2, Nq, Nq, 128, 16, Nq, parents=None)


def test_chain_is_the_chain_of_parents(fa):
    lens, Nq = [5, 200, 131], 9
    par = torch.arange(-1, Nq - 1, dtype=torch.int32).expand(3, Nq).contiguous()
    dev, (o, lse) = run(fa, lens, 4, 2, Nq, Nq, 64, 16, 5, parents=par)
    o2, lse2 = fa.decode_paged_tree(*dev[:5])
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("seed", range(3))
def test_ragged_trees(fa, seed):
    run(fa, [17, 0, 290, 64, 1000], 8, 4, 25, 25, 128, 16, seed, parents="ragged")


def test_several_roots(fa):
    """Trees of their own behind one sequence, and nodes without any tokens before them."""
    par = torch.tensor([[-1, -1, 0, 1, -2, 1, -1, 6], [-2, -1, -1, 2, 3, -2, -2, 1], [-1] * 8], dtype=torch.int32)
    run(fa, [200, 0, 127], 4, 2, 8, 8, 128, 16, 31, parents=par)
    run(fa, [200, 0, 127], 4, 2, 8, 3, 64, 16, 32, parents=par)


def test_long_sequence_is_cut(fa):
    run(fa, [20000], 4, 1, 16, 16, 64, 64, 1)
    run(fa, [9000, 3], 8, 1, 20, 20, 128, 16, 2, parents="ragged")


def test_many_short_sequences(fa):
    lens = [(37 * i) % 90 for i in range(70)]
    run(fa, lens, 8, 4, 6, 6, 64, 16, 3, parents="ragged")


@pytest.mark.parametrize("fill", [float("nan"), float("inf"), -float("inf")])
def test_what_lies_in_unused_places(fa, fill):
    run(fa, [3, 130, 255], 4, 2, 10, 10, 128, 16, 7, fill=fill)
    run(fa, [3, 130, 255], 4, 2, 10, 10, 256, 48, 7, fill=fill, parents="ragged")


@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_hidden_nodes_have_no_influence(fa, value, d):
    """Infinities and NaN in one branch stay with the rows that see it."""
    lens, Nt, page = [126, 40], 12, 16
    k, v, table = make_paged(lens, Nt, page, 2, d, 11)
    par = random_trees(2, Nt, 12)
    for b, n in enumerate(lens):
        for node, c in ((3, 1), (7, d - 1)):
            key = n + node
            v[table[b, key // page], :, key % page, c] = value
        key = n + 5
        k[table[b, key // page], :, key % page, 2] = float("nan")
    q = torch.randn((2, 4, Nt, d), generator=torch.Generator().manual_seed(1)).bfloat16()
    o, lse = fa.decode_paged_tree(*(t.to(DEV) for t in (q, k, v, table, torch.tensor(lens, dtype=torch.int32), par)))
    check_tree(o, lse, oracle_tree(q, k, v, table, lens, par))


def test_largest_and_smallest_scores(fa):
    for scale in (1e-6, 4.0):
        run(fa, [333, 90], 4, 2, 9, 9, 128, 16, 21, scale=scale)
