"""Refusals of the self-tests of the bounded waits, without a GPU (fake addresses)."""
import pytest
import torch

from block_eigenbasis_preconditioning_gb300 import binding

P = 1 << 24


def _norm(rows, dim, *tail):
    return binding.load_library().dobb_selftest_layer_norm_timeout(P, 0, rows, dim, dim, None, None, 0, 1e-5, 8 * P, 0, dim, 16 * P, 17 * P, None, *tail)


def _norm_backward(rows, dim, *tail):
    return binding.load_library().dobb_selftest_layer_norm_backward_timeout(
        P, 0, dim, 8 * P, 0, rows, dim, dim, None, 0, 16 * P, 17 * P, 24 * P, dim, 32 * P, 33 * P, 0, 0, 40 * P, 1 << 26, None, *tail)


def _distill(rows, vocab, *tail):
    return binding.load_library().dobb_selftest_distill_timeout(
        P, 0, rows, vocab, vocab, 8 * P, 4, 9 * P, 0, 3, 1.0, 1.0, 16 * P, 17 * P, 18 * P, 19 * P, 24 * P, vocab, None, None, *tail)


@pytest.mark.parametrize("loaded,limit", [(-1, 1000), (5, 1000), (2, 0), (2, 5 * 10 ** 9 + 1)])
def test_limits(loaded, limit):
    assert _norm(4, 100, loaded, limit) == _norm_backward(4, 100, loaded, limit) == _distill(4, 1000, loaded, 0, limit) == 1
    assert b"loaded_rows" in binding.load_library().dobb_last_error()


def test_calls_without_such_waits():
    if torch.cuda.is_available():
        pytest.skip("made-up addresses")
    assert _norm(4, 16385, 2, 1000) == _norm_backward(4, 11521, 2, 1000) == _distill(4, 300000, 2, 0, 1000) == 6
    for part in (-1, 1, 100):
        assert _distill(4, 1000, 2, part, 1000) == 1 and b"late_part" in binding.load_library().dobb_last_error()
    assert _norm(4, 0, 2, 1000) == _norm_backward(4, 0, 2, 1000) == _distill(4, 0, 2, 0, 1000) == 1
