"""Verification where little is left of the target, against the oracle's exact fractions."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from gpu_common import load_fa
from test_verify_tree_gpu import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    return load_fa()


def truncated(B, V, keep, kids, seed):
    """Targets that are the draft's largest `keep` probabilities made to sum to one, and `kids` drafts
    of other tokens under the root: each rejection leaves a part of what was left, as large as the
    share that was cut off, down to the last places of p - a q."""
    g = np.random.default_rng(seed)
    Nt = 1 + kids
    target, draft = (np.zeros((B, Nt, V), dtype=np.float32) for _ in "pq")
    tokens = np.zeros((B, Nt), dtype=np.int32)
    for b in range(B):
        q = np.exp(g.standard_normal(V))
        q = (q / q.sum()).astype(np.float32)
        out = np.argsort(q)[:-keep]
        p = q.copy()
        p[out] = 0
        target[b], draft[b] = p / p.sum(dtype=np.float64), q
        tokens[b, 1:] = g.choice(out, kids)
    parents = np.zeros((B, Nt), dtype=np.int32)
    parents[:, 0] = -1
    return [torch.from_numpy(x) for x in (tokens, parents, target, draft, g.random((B, Nt)).astype(np.float32))]


@pytest.mark.parametrize("replacement", [True, False])
@pytest.mark.parametrize("keep,kids", [(38, 3), (38, 5), (38, 6), (34, 7), (28, 9)])
def test_truncated_targets(fa, keep, kids, replacement):
    check(fa, *truncated(200, 40, keep, kids, keep + kids), replacement)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_smallest_uniforms(fa, dtype):
    """Uniforms of 2^-45 to 2^-39, each with all its bits, and first tokens of a few 2^-44."""
    B, V = 256, 9
    g = torch.Generator().manual_seed(1)
    target = torch.zeros((B, 1, V))
    target[:, 0, :-1] = torch.randint(0, 4, (B, V - 1), generator=g) * 2.0 ** -44
    target[:, 0, -1] = 1 - 2.0 ** -24
    u = (1 + torch.rand((B, 1), generator=g)) * 2.0 ** -torch.randint(40, 46, (B, 1), generator=g)
    target[0, 0], u[0] = torch.tensor([2.0 ** -44] + [0] * 7 + [1 - 2.0 ** -24]), (1 + 2.0 ** -23) * 2.0 ** -44
    zeros = torch.zeros((B, 1), dtype=torch.int32)
    check(fa, zeros, zeros - 1, target.to(dtype), None, u)
