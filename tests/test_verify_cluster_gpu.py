"""Verification by several CTAs per sequence, sum after sum: many rejections at one node of a large
vocabulary, against the oracle's exact fractions."""
from __future__ import annotations

import pytest
import torch

from gpu_common import load_fa
from spec_common import DEV
from test_verify_tree_gpu import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    return load_fa()


def inputs(B, Nt, V, seed, dtype):
    """Children of the root only, all different and more likely in the draft than in the target, and
    uniforms that reject whatever may be rejected: all of them."""
    g = torch.Generator().manual_seed(seed)
    x = 2 * torch.randn((B, 1, V), generator=g)
    target = torch.softmax(x, -1).to(dtype).expand(B, Nt, V).contiguous()
    draft = torch.softmax(x + torch.randn((B, 1, V), generator=g), -1).to(dtype).expand(B, Nt, V).contiguous()
    parents = torch.zeros((B, Nt), dtype=torch.int32)
    parents[:, 0] = -1
    less = [torch.nonzero(target[b, 0] < draft[b, 0] * (1 - 2.0 ** -6))[:, 0] for b in range(B)]
    tokens = torch.stack([x[torch.randperm(len(x), generator=g)[:Nt]] for x in less]).int()
    u = torch.full((B, Nt), 1 - 2.0 ** -24)
    u[:, 0] = torch.rand(B, generator=g)
    return tokens, parents, target, draft, u


@pytest.mark.parametrize("mode", ["independent", "without", "certain"])
@pytest.mark.parametrize("dtype,V", [(torch.float32, 9001), (torch.float32, 40003), (torch.bfloat16, 70001)])
def test_many_sums_one_after_another(fa, dtype, V, mode):
    """Two and eight CTAs to a sequence."""
    tokens, parents, target, draft, u = inputs(2, 13, V, V, dtype)
    lengths = check(fa, tokens, parents, target, None if mode == "certain" else draft, u, mode != "without")
    assert lengths == [1, 1]


def test_trees_and_sequences_without_one_side_by_side(fa):
    """Clusters that end at once beside ones that go on, in calls right after one another."""
    tokens, parents, target, draft, u = inputs(6, 9, 20000, 3, torch.float32)
    parents[1], parents[4, 0] = -2, 5
    dev = [t.to(DEV) for t in (tokens, parents, target, draft, u)]
    path, new, count = fa.verify_tree(*dev)
    assert fa.fa_device_status() == 7
    assert count[1] == 0 and count[4] == 0 and (path[[1, 4]] == -1).all() and (new[[1, 4]] == -1).all()
    for _ in range(50):
        assert all(torch.equal(a, b) for a, b in zip(fa.verify_tree(*dev), (path, new, count)))
    assert fa.fa_device_status() == 7
    some = [0, 2, 3, 5]
    check(fa, tokens[some], parents[some], target[some], draft[some], u[some])
