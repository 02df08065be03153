"""Stacks whose tiles are too many for one launch go in several groups, each in the same workspace.  (In one group their
momentum was updated before the products were refused.)"""
import ctypes

import pytest

import allreduce_reduction_emulated_gb300 as ar
from allreduce_reduction_emulated_gb300 import _build


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return ar.library()


def test_groups_of_at_most_so_many_tiles(lib):
    def workspace(stacks):
        n = len(stacks)
        counts, rows, cols = ((ctypes.c_size_t * n)(*v) for v in zip(*stacks))
        return lib.ar_orthogonalize_workspace(n, counts, rows, cols, 5)

    # B X of 16 x 2176 is 17 tiles of 64 x 128: 240 stacks of 4096 such matrices are the last below 2^24
    one = (4096, 16, 2176)
    assert 240 * 4096 * 17 <= 1 << 24 < 241 * 4096 * 17
    full = workspace([one] * 240)
    assert full > 239 * 4096 * 16 * 2176 * 2 * 2
    assert workspace([one] * 239) < full
    for more in (241, 256, 300):
        assert workspace([one] * more) == full
    # (17 tiles again) a shape more ends up in the group behind; one stack above the limit is a group of its own
    assert workspace([one] * 240 + [(4096, 17, 2050)]) == full
    large = [(4096, 65536, 520)]
    assert workspace(large + [(1, 200, 200)]) == workspace(large) == workspace([(1, 200, 200)] + large)
