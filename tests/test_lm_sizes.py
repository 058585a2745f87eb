"""Sizes beyond what a call can take are refused, all of them before any device
work, and the arithmetic on them does not overflow (no GPU)."""
import ctypes

import pytest

from block_eigenbasis_preconditioning_gb300 import binding


@pytest.fixture(scope="module")
def lib():
    return binding.load_library()


@pytest.mark.parametrize("numel", [(1 << 63) - 1, (1 << 63) - 16384, (1 << 46), (1 << 45) - 16383])
def test_entries_of_clipping(lib, numel):
    """2^31 - 1 chunks of 16384 entries at most."""
    for sizes in ((numel,), (5, numel, 7)):
        assert lib.dobb_clip_grads_bytes(len(sizes), (ctypes.c_int64 * len(sizes))(*sizes)) == 0
        assert b"too many" in lib.dobb_last_error()
    assert lib.dobb_clip_grads_bytes(1, (ctypes.c_int64 * 1)((1 << 45) - 16384)) > 0
