"""Verification of drafted trees against the oracle's exact fractions: results are equal."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from gpu_common import load_fa
from oracle import spec
from spec_common import DEV, random_trees

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    return load_fa()


def inputs(B, Nt, V, seed, dtype=torch.float32, near=0.7, sharp=2.0, ragged=False):
    """Probabilities of target and draft that resemble each other, drafts drawn at their parents."""
    g = torch.Generator().manual_seed(seed)
    x = sharp * torch.randn((B, Nt, V), generator=g)
    target = torch.softmax(x, -1).to(dtype)
    draft = torch.softmax(x + near * torch.randn((B, Nt, V), generator=g), -1).to(dtype)
    parents = random_trees(B, Nt, seed, ragged)
    up = parents.clamp(min=0).long()
    rows = draft.float().gather(1, up[..., None].expand(B, Nt, V))
    tokens = torch.multinomial(rows.reshape(-1, V), 1, generator=g).reshape(B, Nt).to(torch.int32)
    return tokens, parents, target, draft, torch.rand((B, Nt), generator=g)


def check(fa, tokens, parents, target, draft, uniform, replacement=True):
    dev = [t.to(DEV) if t is not None else None for t in (tokens, parents, target, draft, uniform)]
    path, new, count = (t.cpu() for t in fa.verify_tree(*dev, replacement=replacement))
    assert fa.fa_device_status() == fa.FA_OK
    B, Nt = tokens.shape
    n = [None if t is None else t.double().numpy() for t in (target, draft, uniform)]
    lengths = []
    for b in range(B):
        p, w = spec.verify(tokens[b], None if parents is None else parents[b], n[0][b],
                           None if n[1] is None else n[1][b], n[2][b], replacement)
        assert int(count[b]) == len(p)
        assert path[b].tolist() == p + [-1] * (Nt - len(p))
        assert new[b].tolist() == w + [-1] * (Nt - len(w))
        lengths.append(len(p))
    return lengths


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("mode", ["independent", "without", "certain"])
@pytest.mark.parametrize("Nt,V", [(1, 1), (2, 7), (5, 50), (17, 333), (33, 1001)])
def test_trees(fa, dtype, mode, Nt, V):
    tokens, parents, target, draft, u = inputs(6, Nt, V, Nt + V, dtype, ragged=Nt > 5)
    check(fa, tokens, parents, target, None if mode == "certain" else draft, u, mode != "without")


@pytest.mark.parametrize("V", [4096, 8191, 16385, 40003])
def test_large_vocabularies(fa, V):
    """Several CTAs to a sequence; rows at every alignment."""
    for dtype in (torch.float32, torch.bfloat16):
        tokens, parents, target, draft, u = inputs(2, 5, V, V, dtype)
        check(fa, tokens, parents, target, draft, u)
        check(fa, tokens, parents, target, None, u)


def test_one_cta_and_several_agree(fa):
    """The sums do not depend on how many CTAs share them."""
    t = inputs(3, 9, 20000, 5)
    one = fa.verify_tree(*(x.to(DEV) for x in t))
    many = fa.verify_tree(*(x.repeat((200,) + (1,) * (x.dim() - 1)).to(DEV) for x in t))
    for a, b in zip(one, many):
        assert torch.equal(a.repeat((200,) + (1,) * (a.dim() - 1)), b)


def test_chain(fa):
    tokens, _, target, draft, u = inputs(8, 6, 40, 3, near=0.2)
    chain = torch.arange(-1, 5, dtype=torch.int32).expand(8, 6).contiguous()
    rows = draft[:, [0, 0, 1, 2, 3, 4]]
    tokens = torch.multinomial(rows.reshape(-1, 40), 1, generator=torch.Generator().manual_seed(1)).reshape(8, 6).int()
    assert max(check(fa, tokens, None, target, draft, u)) > 2
    check(fa, tokens, chain, target, draft, u)


def test_many_children_of_one_node(fa):
    """All 255 drafts under the root, most of them rejected one after another."""
    B, Nt, V = 2, 256, 300
    g = torch.Generator().manual_seed(4)
    target = torch.softmax(torch.randn((B, Nt, V), generator=g), -1)
    draft = torch.softmax(torch.randn((B, Nt, V), generator=g), -1)
    parents = torch.zeros((B, Nt), dtype=torch.int32)
    parents[:, 0] = -1
    tokens = torch.randperm(V, generator=g)[:Nt].int().expand(B, Nt).contiguous()
    u = torch.full((B, Nt), 1 - 2.0 ** -24)  # rejects whatever may be rejected
    for replacement in (True, False):
        check(fa, tokens, parents, target, draft, u, replacement)
    check(fa, tokens, parents, target, None, u)


def test_equal_distributions_accept_everything(fa):
    tokens, parents, target, _, u = inputs(4, 8, 64, 9)
    lengths = check(fa, tokens, parents, target, target.clone(), u)
    assert all(n > 1 for n in lengths)


def test_drafts_that_leave_nothing(fa):
    """Certain drafts of all that has any probability, and a draft row that covers the target's."""
    B, Nt, V = 2, 4, 8
    target = torch.zeros((B, Nt, V))
    target[..., 2], target[..., 5] = 0.5, 0.25  # sums to less than one: u = 3/4 rejects both
    parents = torch.tensor([[-1, 0, 0, -2]] * B, dtype=torch.int32)
    tokens = torch.tensor([[0, 2, 5, 0]] * B, dtype=torch.int32)
    u = torch.full((B, Nt), 0.75)
    check(fa, tokens, parents, target, None, u)
    draft = torch.zeros_like(target)
    draft[..., 2], draft[..., 5] = 0.75, 0.5
    check(fa, tokens, parents, target, draft, u)


def test_rows_without_probability(fa):
    target = torch.zeros((2, 3, 16))
    parents = torch.tensor([[-1, 0, 0], [-2, -2, -2]], dtype=torch.int32)
    tokens = torch.ones((2, 3), dtype=torch.int32)
    path, new, count = fa.verify_tree(*(t.to(DEV) for t in (tokens, parents, target)), None,
                                      torch.rand((2, 3)).to(DEV))
    assert path.tolist() == [[0, -1, -1], [-1, -1, -1]]
    assert new.tolist() == [[-1, -1, -1], [-1, -1, -1]] and count.tolist() == [1, 0]


@pytest.mark.parametrize("u0", [0.0, 0.5, 1 - 2.0 ** -24, 1.0, float("nan")])
def test_ends_of_the_unit_interval(fa, u0):
    """The first and last tokens that have a probability; numbers out of range stay in the row."""
    V = 5000
    target = torch.zeros((1, 1, V))
    target[0, 0, 100], target[0, 0, 4000] = 0.5, 0.5
    _, new, count = fa.verify_tree(torch.zeros((1, 1), dtype=torch.int32, device=DEV), None, target.to(DEV), None,
                                   torch.full((1, 1), u0, device=DEV))
    assert new.item() == (100 if not u0 >= 0.5 else 4000) and count.item() == 1


def test_nan_and_negative_values_count_as_zero(fa):
    tokens, parents, target, draft, u = inputs(3, 6, 100, 13)
    clean_t, clean_d = target.clone(), draft.clone()
    target[:, :, 7], clean_t[:, :, 7] = float("nan"), 0.0
    target[:, :, 11], clean_t[:, :, 11] = -0.5, 0.0
    draft[:, :, 13], clean_d[:, :, 13] = float("nan"), 0.0
    bad = [t.to(DEV) for t in (tokens, parents, target, draft, u)]
    good = [t.to(DEV) for t in (tokens, parents, clean_t, clean_d, u)]
    for a, b in zip(fa.verify_tree(*bad), fa.verify_tree(*good)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("replacement", [True, False])
def test_first_token_has_the_targets_distribution(fa, replacement):
    """Of 2^17 sequences with three drafts each, the first new token's counts are the target's
    probabilities to within 6 standard deviations."""
    B, Nt, V = 1 << 17, 4, 12
    g = torch.Generator(device=DEV).manual_seed(2)
    p = torch.softmax(torch.randn(V, generator=g, device=DEV), -1)
    q = torch.softmax(torch.randn(V, generator=g, device=DEV), -1)
    tokens = torch.multinomial(q.expand(B, V), 3, replacement=replacement, generator=g).int()
    tokens = torch.cat((torch.zeros((B, 1), dtype=torch.int32, device=DEV), tokens), 1).contiguous()
    parents = torch.tensor([-1, 0, 0, 0], dtype=torch.int32, device=DEV).expand(B, Nt).contiguous()
    u = torch.rand((B, Nt), generator=g, device=DEV)
    _, new, _ = fa.verify_tree(tokens, parents, p.expand(B, Nt, V).contiguous(), q.expand(B, Nt, V).contiguous(), u,
                               replacement=replacement)
    n = torch.bincount(new[:, 0].long(), minlength=V).double().cpu().numpy()
    p = p.double().cpu().numpy()
    assert np.all(np.abs(n - B * p) <= 6 * np.sqrt(B * p * (1 - p)) + 1)


def test_bad_trees_are_refused_one_by_one(fa):
    tokens, parents, target, draft, u = inputs(5, 6, 50, 17)
    good = [t.to(DEV) for t in (tokens, parents, target, draft, u)]
    ref = fa.verify_tree(*good)
    parents, tokens = parents.clone(), tokens.clone()
    parents[0, 3] = 3                       # its own parent
    parents[1, 2], parents[1, 4] = -2, 2    # below a missing node
    tokens[3, 5] = 50                       # no such token
    parents[4, 2] = -1                      # a second root
    path, new, count = fa.verify_tree(tokens.to(DEV), parents.to(DEV), *good[2:])
    assert fa.fa_device_status() == 7
    for b in (0, 1, 3, 4):
        assert count[b] == 0 and (path[b] == -1).all() and (new[b] == -1).all()
    for a, r in zip((path, new, count), ref):
        assert torch.equal(a[2], r[2])
