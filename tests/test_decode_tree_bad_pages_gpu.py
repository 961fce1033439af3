"""A bad page is seen wherever it lies in a tile, whichever lane of the copying warp looks it up."""
from __future__ import annotations

import pytest
import torch

from gpu_common import load_fa
from spec_common import DEV, make_paged, random_trees

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    return load_fa()


@pytest.mark.parametrize("H,Hkv,d", [(4, 2, 64), (40, 1, 128), (2, 1, 256)])
@pytest.mark.parametrize("page", [1, 4, 16, 64])
def test_every_place_of_a_bad_page(fa, page, H, Hkv, d):
    lens, Nt = [200, 63], 4
    k, v, table = make_paged(lens, Nt, page, Hkv, d, page)
    q = torch.randn((2, H, Nt, d), generator=torch.Generator().manual_seed(1)).bfloat16().to(DEV)
    k, v, n, par = (t.to(DEV) for t in (k, v, torch.tensor(lens, dtype=torch.int32), random_trees(2, Nt, 2)))
    good = table.to(DEV)
    ref = fa.decode_paged_tree(q, k, v, good, n, par)[0]
    assert fa.fa_device_status() == fa.FA_OK
    for b, length in enumerate(lens):
        for at in range(-(-(length + Nt) // page)):
            bad, out, lse = good.clone(), torch.full_like(q, 7.0), torch.full(q.shape[:3], 7.0, device=DEV)
            bad[b, at] = -1 if at % 2 else k.shape[0]
            fa.decode_paged_tree(q, k, v, bad, n, par, out=out, lse=lse)
            assert fa.fa_device_status() == 7, (b, at)
            assert (out[b] == 7).all() and (lse[b] == 7).all(), (b, at)
            # (the work is cut by lengths alone, so the other sequence keeps its bits)
            assert torch.equal(out[1 - b], ref[1 - b]), (b, at)
