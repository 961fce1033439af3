"""Pages of kept rows that are already in their places are looked at like those of rows that move."""
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


@pytest.mark.parametrize("page", [-1, 1000])
def test_bad_pages_of_rows_that_stay(fa, page):
    """Sequences whose rows all stay, whose first rows stay, and which lie on other pages."""
    lens, Nt = [10, 12, 15, 30, 14, 14], 6
    k, v, table = make_paged(lens, Nt, 16, 2, 64, 3, width=3)
    path = torch.tensor([[0, 1, 2, -1, -1, -1], [0, 1, 2, 3, 5, -1], [0, 1, 3, -1, -1, -1],
                         [0, 2, -1, -1, -1, -1], [0, 1, 2, -1, -1, -1], [0, 1, -1, -1, -1, -1]], dtype=torch.int32)
    count = torch.tensor([3, 5, 3, 2, 3, 2], dtype=torch.int32)
    table[0, 0] = page  # rows 10, 11, 12 stay
    table[1, 0] = page  # rows 12 to 15 stay there, the row that moves is on the next page
    table[2, 0] = page  # row 15 stays there
    table[3, 0] = page  # rows 30 and 31: not its page
    table[4, 1] = page  # row 16 stays there
    table[5, 1] = page  # rows 14 and 15: not its page
    n = torch.tensor(lens, dtype=torch.int32)
    dev = [k.to(DEV), v.to(DEV)]
    out = fa.keep_path(dev, *(t.to(DEV) for t in (table, n, path, count)))
    assert fa.fa_device_status() == 7
    assert out.tolist() == [10, 12, 15, 32, 14, 16]
    for c, got in zip((k, v), dev):
        want = spec.keep(c.view(torch.int16).numpy(), table.numpy(), lens, path.numpy(), [0, 0, 0, 2, 0, 2])
        assert np.array_equal(got.cpu().view(torch.int16).numpy(), want)
