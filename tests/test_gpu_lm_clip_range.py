"""Clipping where sums of squares, factors and stretches of chunks leave the
ordinary: against the fp64 definition on the same data.

A thread sums 32 squares in four fp32 chains of eight and joins them (11
roundings u of a positive sum), adds the result to an fp32 pair (n partial sums: n^2 u^2
of the sum, below u for n < 4096) or in fp64, and all else is fp64: a sum of
squares is off by at most 12 u of itself, its root by 6 u, the norm's fp32 value by one
more rounding.  The factor is off by 6 u and its own rounding, a scaled entry by two
more roundings and the output's."""
import pytest
import torch

from lm_util import HALF_UNIT, TORCH, U

pytestmark = pytest.mark.gpu

NORM = 8 * U


def _dobb():
    import block_eigenbasis_preconditioning_gb300 as d
    return d


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("value,numel", [(3e18, 16384), (3e18, 70001), (2.5e18, 64), (1.2e17, 1 << 29), (5e17, 120000001), (1e14, 1 << 28)])
def test_squares_whose_sums_near_the_end_of_fp32(dtype, value, numel):
    """Each group of 32 squares is within fp32, the sum of the groups of one
    thread is not."""
    g = torch.full((numel,), value, device="cuda", dtype=TORCH[dtype])
    small = torch.ones(77, device="cuda", dtype=TORCH[dtype])
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = _dobb().grad_norm([small, g], flags=flags)
    want = float(g[0]) * numel ** 0.5
    assert int(flags) == 0
    assert abs(float(r.norm) - want) <= NORM * want and abs(float(r.norms[1]) - want) <= NORM * want
    assert abs(float(r.norms[0]) - 77 ** 0.5) <= NORM * 77 ** 0.5
    outs = [torch.empty_like(small), torch.empty_like(g)]
    r = _dobb().clip_grads([small, g], 1.0, out=outs, flags=flags)
    assert int(flags) == 0
    entry = float(g[0]) / want
    assert float(outs[1].min()) == float(outs[1].max())
    assert abs(float(outs[1][0]) - entry) <= (NORM + 2 * U + HALF_UNIT[dtype] * 1.001) * entry
