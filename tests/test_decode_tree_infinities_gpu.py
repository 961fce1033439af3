"""Infinite values of nodes whose probabilities are far below fp32's range, in items that were cut: the
nodes lie in a part of their own, which weighs nothing beside the cached tokens'."""
from __future__ import annotations

import pytest
import torch

from gpu_common import load_fa
from spec_common import DEV, check_tree, make_paged, oracle_tree, random_trees

pytestmark = pytest.mark.gpu

INF = float("inf")


@pytest.fixture(scope="module")
def fa():
    return load_fa()


def inputs(length, H, Nt, d, seed):
    """One sequence of whole tiles (a tile per CTA: fewer than 150 in all); the cached tokens' scores
    lie 110 above the nodes', so the nodes weigh e^-110."""
    k, v, table = make_paged([length], Nt, 64, 1, d, seed)
    q = torch.randn((1, H, Nt, d), generator=torch.Generator().manual_seed(seed)).bfloat16()
    q[..., 0] = 8.0
    for key in range(length + Nt):
        k[table[0, key // 64], :, key % 64, 0] = 110 * d ** 0.5 / 8 if key < length else 0.0
    return q, k, v, table, torch.tensor([length], dtype=torch.int32)


def put(v, table, key, column, value):
    v[table[0, key // 64], :, key % 64, column] = value


@pytest.mark.parametrize("length,H,Nt,d", [(12800, 4, 16, 64), (6400, 2, 9, 96), (12800, 16, 16, 128), (6400, 3, 12, 256),
                                           (3712, 64, 20, 128), (896, 80, 16, 256)])
def test_nodes_that_weigh_nothing(fa, length, H, Nt, d):
    """Few rows and many, merged by rows and by the list of cuts."""
    q, k, v, table, lens = inputs(length, H, Nt, d, d + Nt)
    par = random_trees(1, Nt, Nt)
    for node, column, value in ((3, 1, INF), (5, 2, -INF), (0, 4, INF), (7, 4, -INF), (2, d - 1, float("nan")), (0, 33, -INF)):
        put(v, table, length + node, column, value)
    ref = oracle_tree(q, k, v, table, [length], par)
    o, lse = fa.decode_paged_tree(*(t.to(DEV) for t in (q, k, v, table, lens, par)))
    assert fa.fa_device_status() == fa.FA_OK
    assert (o[..., 33] == -INF).all() and o[..., 4].isnan().any() and (o[..., 1] == INF).any()
    check_tree(o, lse, ref)


@pytest.mark.parametrize("length", [0, 100, 12800])
def test_a_node_with_a_score_of_minus_infinity(fa, length):
    """It has no weight at all; its infinity is the column's whether it has a part of its own or not."""
    q, k, v, table, lens = inputs(length, 4, 1, 64, 5)
    finite = oracle_tree(q, k, v, table, [length], None)
    k[table[0, length // 64], :, length % 64, 0] = -INF
    put(v, table, length, 40, INF)
    o, lse = fa.decode_paged_tree(*(t.to(DEV) for t in (q, k, v, table, lens)))
    assert fa.fa_device_status() == fa.FA_OK
    assert (o[..., 40] == INF).all()
    o[..., 40] = 0
    if length:  # the cached tokens' result, which the node with its e^-110 left as it was
        finite[0][..., 40] = 0
        check_tree(o, lse, finite)
    else:
        assert (o == 0).all() and (lse == -INF).all()
