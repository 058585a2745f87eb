"""Layer norm's launches, of every width: their shared memory is what a launch may ask for.  No GPU."""
import ctypes

import pytest

from block_eigenbasis_preconditioning_gb300 import binding

F32, BF16 = 0, 1


@pytest.mark.parametrize("rows", [1, 8, 152, 153, 304, 305, 2000, 100000])
@pytest.mark.parametrize("backward,last", [(0, 16384), (1, 11520)])
def test_the_shared_memory_of_every_width(rows, backward, last):
    smem, most = binding.load_library().dobb_selftest_layer_norm_smem, ctypes.c_int64()
    for x, g in ((F32, F32), (BF16, BF16), (F32, BF16)):
        for dim in range(1, last + 1):
            for gap in (0, 1):
                n = smem(rows, dim, x, dim + gap, g, dim + gap, backward, ctypes.byref(most))
                assert 0 < n <= most.value, (rows, dim, x, g, gap, n)
        assert smem(rows, last + 1, x, last + 1, g, last + 1, backward, None) == 0
    # (an SM gives a block 227 KB; the barriers and the joins' numbers lie beside this)
    assert most.value <= 226 * 1024


def test_sizes_that_are_refused():
    smem = binding.load_library().dobb_selftest_layer_norm_smem
    for args in ((0, 5, 0, 5, 0, 5), (-1, 5, 0, 5, 0, 5), (2, 0, 0, 5, 0, 5), (2, 5, 2, 5, 0, 5), (2, 5, 0, 4, 0, 5), (2, 5, 0, 5, 0, 4)):
        assert smem(*args, 0, None) == -1
