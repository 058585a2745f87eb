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


@pytest.mark.parametrize("count,dim", [(4, (1 << 63) - 1), (4, 1 << 62), (1, 1 << 41), ((1 << 31) - 1, 1 << 15), ((1 << 31) - 1, 1 << 40),
                                       ((1 << 31) - 1, 1 << 52), (1 << 20, 1 << 26)])
def test_tokens_and_columns_of_the_embedding(lib, count, dim):
    """The blocks of the gradient's last kernel are 2^31 - 1 at most: refused by
    the workspace's size already, and by the call before its first launch."""
    assert lib.dobb_embedding_backward_bytes(count, 100, dim) == 0 and b"too many" in lib.dobb_last_error()
    p = 1 << 20
    assert lib.dobb_embedding_backward(p, 0, count, dim, dim, p, 8, 1, 1.0, p, 0, dim, 0, None, p, 1 << 62, None) == 6
    assert b"too many" in lib.dobb_last_error()


def test_columns_of_the_lookup(lib):
    p = 1 << 20
    for dim in ((1 << 63) - 1, (1 << 63) - 9, 1 << 61):
        assert lib.dobb_embedding(p, 1, 1, dim, dim, p, 8, 1 << 40, 1.0, p, 1, dim, None, None) in (1, 6)
