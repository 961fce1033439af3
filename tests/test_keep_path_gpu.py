"""Keeping the accepted nodes' rows of a paged bf16 cache: the bytes of the oracle."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from gpu_common import load_fa
from oracle import spec
from spec_common import DEV, make_paged

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    return load_fa()


def paths(B, Nt, seed, share=0.4):
    g = np.random.default_rng(seed)
    path, count = np.full((B, Nt), -1, dtype=np.int32), np.zeros(B, dtype=np.int32)
    for b in range(B):
        take = np.flatnonzero(g.random(Nt) < share)
        path[b, :len(take)], count[b] = take, len(take)
    return torch.from_numpy(path), torch.from_numpy(count)


def check(fa, lens, Nt, page, Hkv, d, layers, path, count, seed=1):
    caches, table = [], None
    for i in range(layers):
        k, v, table = make_paged(lens, Nt, page, Hkv, d, seed)
        g = torch.Generator().manual_seed(seed + 10 * i)
        caches += [torch.randn(k.shape, generator=g).bfloat16(), v]
    dev = [c.to(DEV) for c in caches]
    n = torch.tensor(lens, dtype=torch.int32)
    out = fa.keep_path(dev, table.to(DEV), n.to(DEV), path.to(DEV), count.to(DEV))
    assert fa.fa_device_status() == fa.FA_OK
    assert torch.equal(out.cpu(), n + count)
    for c, got in zip(caches, dev):
        want = spec.keep(c.view(torch.int16).numpy(), table.numpy(), lens, path.numpy(), count.numpy())
        assert np.array_equal(got.cpu().view(torch.int16).numpy(), want)


@pytest.mark.parametrize("d", [64, 96, 128, 256])
@pytest.mark.parametrize("page", [1, 7, 16, 48])
def test_rows(fa, d, page):
    path, count = paths(5, 23, d + page)
    check(fa, [0, 1, 15, 100, 333], 23, page, 3, d, 2, path, count)


@pytest.mark.parametrize("Nt,share", [(1, 1.0), (2, 0.5), (64, 0.1), (256, 0.5), (256, 0.95), (256, 1.0)])
def test_paths(fa, Nt, share):
    """Short and long paths, ones that move nothing, and moves that overlap."""
    path, count = paths(3, Nt, Nt, share)
    check(fa, [9, 0, 40], Nt, 16, 2, 128, 1, path, count)


def test_every_row_moves_by_one(fa):
    path = torch.cat((torch.arange(1, 256), torch.tensor([-1]))).int().expand(2, 256).contiguous()
    check(fa, [5, 33], 256, 16, 2, 64, 1, path, torch.tensor([255, 200], dtype=torch.int32))


def test_nothing_kept(fa):
    path, count = torch.full((2, 4), -1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    check(fa, [9, 0], 4, 16, 2, 128, 2, path, count)


def test_many_layers_and_sequences(fa):
    path, count = paths(40, 12, 5)
    check(fa, [(7 * i) % 50 for i in range(40)], 12, 16, 4, 64, 9, path, count)


def test_bad_sequences_are_left_as_they_are(fa):
    lens, Nt = [10, 20, 30, 40, 50, 60], 8
    k, _, table = make_paged(lens, Nt, 16, 2, 64, 3)
    path = torch.tensor([[0, 2, 5, -1, -1, -1, -1, -1]] * 6, dtype=torch.int32)
    count = torch.tensor([3, 3, 9, 3, 3, 3], dtype=torch.int32)
    path[0, 2] = 2                   # not ascending
    path[1, 2] = 8                   # no such node
    n = torch.tensor(lens, dtype=torch.int32)
    n[3] = -1
    table[4, (50 + 5) // 16] = 1000  # page of a moved row
    dev, old = k.to(DEV), k.clone()
    out = fa.keep_path([dev], *(t.to(DEV) for t in (table, n, path, count)))
    assert fa.fa_device_status() == 7
    want = spec.keep(old.view(torch.int16).numpy(), table.numpy(), n.numpy(), path.numpy(), [0, 0, 0, 0, 0, 3])
    assert np.array_equal(dev.cpu().view(torch.int16).numpy(), want)
    assert out.tolist() == [10, 20, 30, -1, 50, 63]
