"""The global gradient norm and clipping on the GPU against the fp64
definition.  Squares are summed in fp32 chains of at most 256 additions and
joined in fp64 (or wider throughout): a sum of squares is off by at most
256 u of itself, its root by half of that, so the norm and the factor by
130 u; a scaled entry by 132 u of itself and one rounding."""
import numpy as np
import pytest
import torch

from oracle import lm as L

from lm_util import HALF_UNIT, TINY, TORCH, U, np64, rounded

pytestmark = pytest.mark.gpu

NORM = 130 * U


def _dobb():
    import block_eigenbasis_preconditioning_gb300 as d
    return d


def _view(x, dtype, offset):
    buf = torch.empty(x.size + offset, dtype=TORCH[dtype], device="cuda")
    v = buf[offset:].view(x.shape)
    v.copy_(torch.from_numpy(x).cuda())
    return v


def _check(xs, gds, odts, max_norm, r, outs):
    norm, c, norms, want = L.clip_grads(xs, max_norm)
    near = lambda got, want: got == np.inf if want > np.finfo(np.float32).max else abs(got - want) <= NORM * want + TINY["f32"]  # noqa: E731
    assert near(float(r.norm), norm)
    assert abs(float(r.scale) - c) <= (NORM + U) * c
    assert all(near(a, b) for a, b in zip(np64(r.norms), norms))
    for w, o, dt in zip(want, outs, odts):
        assert (np.abs(np64(o) - w) <= (NORM + 2 * U + HALF_UNIT[dt] * 1.001) * np.abs(w) + TINY[dt]).all()


SETS = [
    [(1,)],
    [(7,), (1, 1), (33, 3)],
    [(768, 768)],
    [(1000, 1001), (5,), (0,), (64, 64), (32768,), (32769,), (2, 16384)],
    [(0,), (3, 0)],
    [(3,)] * 1100 + [(70001,)],           # more tensors than one launch's table
]


@pytest.mark.parametrize("gdt", ["f32", "bf16", "mixed"])
@pytest.mark.parametrize("odt", ["f32", "bf16", "mixed"])
@pytest.mark.parametrize("which", range(len(SETS)))
@pytest.mark.parametrize("offset", [0, 1])
def test_norm_and_clip(gdt, odt, which, offset):
    shapes = SETS[which]
    rng = np.random.default_rng(which)
    pick = lambda d, i: d if d != "mixed" else ("f32", "bf16")[(i + (d == odt)) % 2]  # noqa: E731
    gds, odts = [pick(gdt, i) for i in range(len(shapes))], [pick(odt, i + 1) for i in range(len(shapes))]
    xs = [rounded(rng.standard_normal(s) * 10.0 ** rng.uniform(-4, 1), d) for s, d in zip(shapes, gds)]
    gs = [_view(x, d, offset * (i % 3)) for i, (x, d) in enumerate(zip(xs, gds))]
    kept = [g.clone() for g in gs]
    for max_norm in (0.5, 1e9, 0.0):
        outs = [torch.empty(g.numel() + offset, dtype=TORCH[d], device="cuda")[offset:].view(g.shape) for g, d in zip(gs, odts)]
        flags = torch.zeros(1, dtype=torch.int32, device="cuda")
        r = _dobb().clip_grads(gs, max_norm, out=outs, flags=flags)
        _check(xs, gds, odts, max_norm, r, outs)
        assert int(flags) == 0 and all(torch.equal(a, b) for a, b in zip(gs, kept))
        assert torch.equal(r.norm, _dobb().grad_norm(gs).norm)
    assert float(_dobb().grad_norm(gs).scale) == 1.0
    r = _dobb().clip_grads(gs, 0.25)       # in place
    _check(xs, gds, gds, 0.25, r, gs)


@pytest.mark.parametrize("seed", range(4))
@pytest.mark.parametrize("count", [12, 400, 900])
def test_small_tensors_side_by_side(seed, count):
    """Small tensors, empty ones and longer ones in any order, types and
    alignments: neighbours of up to a few thousand entries are taken together."""
    rng = np.random.default_rng(1000 * seed + count)
    sizes = rng.choice([0, 0, 1, 7, 8, 9, 768, 1024, 4095, 4096, 4097, 16384, 16385, 40000], count,
                       p=[0.07] * 2 + [0.08] * 10 + [0.03] * 2)
    gds, odts = rng.choice(["f32", "bf16"], (2, count))
    xs = [rounded(rng.standard_normal(n) * 10.0 ** rng.uniform(-3, 1), d) for n, d in zip(sizes, gds)]
    gs = [_view(x, d, int(o)) for x, d, o in zip(xs, gds, rng.integers(0, 5, count))]
    outs = [_view(np.zeros(n), d, int(o)) for n, d, o in zip(sizes, odts, rng.integers(0, 5, count))]
    r = _dobb().clip_grads(gs, 0.75, out=outs)
    _check(xs, gds, odts, 0.75, r, outs)
    r = _dobb().clip_grads(gs, 1e9, out=outs)
    _check(xs, gds, odts, 1e9, r, outs)
    q = _dobb().grad_norm(gs)
    assert torch.equal(q.norms, r.norms) and torch.equal(q.norm, r.norm)
    r = _dobb().clip_grads(gs, 0.75)
    _check(xs, gds, gds, 0.75, r, gs)


@pytest.mark.parametrize("gdt", ["f32", "bf16"])
@pytest.mark.parametrize("size", [1e-30, 3e-23, 1e15, 2e19, 1e37])
def test_squares_outside_the_range_of_fp32(gdt, size):
    """Entries whose squares underflow or overflow fp32, next to ordinary ones."""
    rng = np.random.default_rng(3)
    xs = [rounded(rng.standard_normal(s) * a, gdt) for s, a in (((300, 70),  size), ((50,), 1.0 if size > 1 else size), ((40000,), size))]
    gs = [torch.from_numpy(x).cuda().to(TORCH[gdt]) for x in xs]
    outs = [torch.empty_like(g, dtype=torch.float32) for g in gs]
    max_norm = float(L.clip_grads(xs, 1.0)[0]) / 3
    r = _dobb().clip_grads(gs, max_norm, out=outs)
    _check(xs, [gdt] * 3, ["f32"] * 3, float(np.float32(max_norm)), r, outs)
    one = xs[0].copy()
    one[:] = 0
    one[7, 3] = xs[0][7, 3]                # a single tiny or huge entry among zeros
    r = _dobb().grad_norm([torch.from_numpy(one).cuda().to(TORCH[gdt])])
    assert abs(float(r.norm) - abs(one[7, 3])) <= NORM * abs(one[7, 3]) + TINY["f32"]


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("gdt", ["f32", "bf16"])
def test_non_finite_gradients_are_passed_on(bad, gdt):
    xs = [np.ones((40, 50), np.float32), np.ones(70000, np.float32)]
    xs[1][69999] = bad
    gs = [torch.from_numpy(x).cuda().to(TORCH[gdt]) for x in xs]
    outs = [torch.zeros_like(g) for g in gs]
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = _dobb().clip_grads(gs, 1.0, out=outs, flags=flags)
    assert int(flags) == 2 and float(r.scale) == 1.0 and not np.isfinite(float(r.norm))
    assert abs(float(r.norms[0]) - 2000 ** 0.5) <= NORM * 2000 ** 0.5 and not np.isfinite(float(r.norms[1]))
    for g, o in zip(gs, outs):
        assert torch.equal(g.nan_to_num(5.0, 6.0, 7.0), o.nan_to_num(5.0, 6.0, 7.0))
    _dobb().clip_grads(gs, 1.0)
    assert float(gs[0].float().sum()) == 2000.0


def test_orders_of_dimensions_and_a_side_stream():
    g = torch.randn(30, 40, 5, device="cuda")
    t = g.permute(2, 0, 1)
    want = float(g.double().norm())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    r = _dobb().clip_grads([t], 1.0, stream=side)
    side.synchronize()
    assert abs(float(r.norm) - want) <= NORM * want
    assert abs(float(g.double().norm()) - 1.0) <= 300 * U
    # clipped already: the factor is 1 within rounding, and the norm stays
    r = _dobb().clip_grads([g], 1.0 + 1e-3)
    assert float(r.scale) == 1.0


def test_more_entries_than_32_bits_index():
    n = (1 << 31) + 5
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g[0], g[n - 1], g[(1 << 31) - 1] = 3.0, 4.0, 12.0
    r = _dobb().clip_grads([g], 1.0)
    assert abs(float(r.norm) - 13.0) <= NORM * 13.0
    assert float(g[n - 1]) == float(torch.tensor(4.0 / 13).bfloat16()) and float(g[0]) == float(torch.tensor(3.0 / 13).bfloat16())
