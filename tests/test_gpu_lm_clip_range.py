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

from lm_util import HALF_UNIT, TINY, TORCH, U

pytestmark = pytest.mark.gpu

NORM = 8 * U
FP32_MAX = float(torch.finfo(torch.float32).max)


def _dobb():
    import block_eigenbasis_preconditioning_gb300 as d
    return d


def _check(gs, max_norm, r, outs):
    norms = torch.stack([g.double().square().sum().sqrt() for g in gs])
    norm = float(norms.square().sum().sqrt())
    c = max_norm / norm if norm > max_norm else 1.0
    near = lambda got, want: got == float("inf") if want > FP32_MAX else abs(got - want) <= NORM * want + TINY["f32"]  # noqa: E731
    assert near(float(r.norm), norm), (float(r.norm), norm)
    assert abs(float(r.scale) - c) <= NORM * c + TINY["f32"]
    assert all(near(float(a), float(b)) for a, b in zip(r.norms, norms))
    for g, o in zip(gs, outs):
        dt = "bf16" if o.dtype == torch.bfloat16 else "f32"
        want = g.double() * c
        bound = (NORM + 2 * U + HALF_UNIT[dt] * 1.001) * want.abs() + TINY[dt]
        assert bool(((o.double() - want).abs() <= bound).all())


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


@pytest.mark.parametrize("gdt,odt,in_place", [("f32", "f32", False), ("f32", "bf16", False), ("bf16", "f32", False), ("bf16", "bf16", False),
                                              ("f32", "f32", True), ("bf16", "bf16", True)])
@pytest.mark.parametrize("size,max_norm", [(1e37, 1e-3), (1e37, 1e-5), (3e38, 1e-7), (2e36, 7.0), (1e37, 1e-44)])
def test_factors_below_the_normal_range_of_fp32(gdt, odt, in_place, size, max_norm):
    gen = torch.Generator(device="cuda").manual_seed(5)
    R = lambda *s: (torch.rand(*s, device="cuda", generator=gen) * 2 - 1) * size  # noqa: E731
    gs = [R(300, 401).to(TORCH[gdt]), R(7).to(TORCH[gdt]), R(5).to(TORCH[gdt]), R(40001).to(TORCH[gdt])[1:]]
    kept = [g.clone() for g in gs]
    outs = gs if in_place else [torch.empty_like(g, dtype=TORCH[odt]) for g in gs]
    r = _dobb().clip_grads(gs, max_norm, out=None if in_place else outs)
    _check(kept, float(torch.tensor(max_norm)), r, outs)


@pytest.mark.parametrize("gdt", ["f32", "bf16", "mixed"])
@pytest.mark.parametrize("odt", ["f32", "bf16"])
def test_many_chunks_per_block(gdt, odt):
    """Tensors over many chunks and over several blocks' stretches, odd sizes
    and offsets, with entries of very different size along the way."""
    gen = torch.Generator(device="cuda").manual_seed(6)
    gs = []
    for i, s in enumerate([(9001, 1601), (3,), (20000003,), (768,), (8000009,)]):
        dt = TORCH[gdt if gdt != "mixed" else ("f32", "bf16")[i % 2]]
        n = 1
        for k in s:
            n *= k
        buf = torch.randn(n + i, device="cuda", generator=gen)
        buf *= torch.exp(3.0 * torch.sin(torch.arange(n + i, device="cuda") * (6.0 / n)))
        gs.append(buf.to(dt)[i:].view(s))
    kept = [g.clone() for g in gs]
    outs = [torch.empty(g.numel() + 1, device="cuda", dtype=TORCH[odt])[1:].view(g.shape) for g in gs]
    for max_norm in (0.5, 1e9):
        r = _dobb().clip_grads(gs, max_norm, out=outs)
        _check(kept, max_norm, r, outs)
        q = _dobb().clip_grads(gs, max_norm, out=outs)
        assert torch.equal(r.norms, q.norms) and torch.equal(r.norm, q.norm)
    r = _dobb().clip_grads(gs, 0.5)
    _check(kept, 0.5, r, gs)
