"""Cache buffers that overlap are refused: a row moved in both would follow its own place."""
import ctypes

import pytest

from test_boundary_cpu import fa  # noqa: F401
from test_spec_cpu import KEEP, P

SIZE = KEEP["num"] * KEEP["Hkv"] * KEEP["ps"] * KEEP["d"] * 2


@pytest.mark.parametrize("caches,code", [
    ((P, P), 1), ((P, P + 16), 1), ((P, P + SIZE - 16), 1), ((P + SIZE - 16, P), 1),
    ((P, P + 2 * SIZE, P + SIZE + 16), 1),
    # side by side they pass, and the next argument is looked at (here: not aligned)
    ((P, P + SIZE), 3), ((P + 2 * SIZE, P, P + SIZE), 3),
])
def test_overlapping_caches(fa, caches, code):  # noqa: F811
    a = {**KEEP, "caches": (ctypes.c_void_p * len(caches))(*caches), "n": len(caches), "path": P + 2}
    assert fa.fa_keep_path(*a.values()) == code
