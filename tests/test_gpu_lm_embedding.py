"""The embedding lookup and its gradient on the GPU against the fp64
definitions.  The lookup is one fp32 product rounded once: equal bit for bit.
A row's gradient is a sum of c terms in fp32 in some fixed order, off by at
most (c + 3) u times the sum of the terms' absolute values, and rounded once."""
import numpy as np
import pytest
import torch

from oracle import lm as L

from lm_util import HALF_UNIT, TINY, TORCH, U, dev, np64, rounded, strided

pytestmark = pytest.mark.gpu


def _dobb():
    import block_eigenbasis_preconditioning_gb300 as d
    return d


@pytest.mark.parametrize("wdt", ["f32", "bf16"])
@pytest.mark.parametrize("odt", ["f32", "bf16"])
@pytest.mark.parametrize("count,dim,extra,offset", [(1, 1, 0, 0), (1, 1600, 0, 0), (3, 7, 1, 1), (17, 129, 3, 5), (300, 64, 0, 8),
                                                    (5, 4096, 8, 0), (1000, 33, 0, 0)])
@pytest.mark.parametrize("scale", [1.0, 1.7])
def test_lookup(wdt, odt, count, dim, extra, offset, scale):
    vocab = 211
    rng = np.random.default_rng(count + dim)
    w = rounded(rng.standard_normal((vocab, dim)), wdt)
    t = rng.integers(-2, vocab + 1, count)
    t[0] = vocab - 1
    wd = strided(w, wdt, extra, offset)
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    for tdt in (torch.int64, torch.int32):
        td = torch.from_numpy(t).to("cuda", tdt)
        got = _dobb().embedding(wd, td, scale=scale, out_dtype=TORCH[odt], flags=flags)
        live = torch.from_numpy((t >= 0) & (t < vocab)).cuda()[:, None]
        want = torch.where(live, dev(w, wdt)[td.clamp(0, vocab - 1).long()].float() * scale, 0.0).to(TORCH[odt])
        assert torch.equal(got, want)
        o = strided(np.zeros((count, dim)), odt, 5, 3)
        _dobb().embedding(wd, td, scale=scale, out=o)
        assert torch.equal(o, want)
        assert torch.isnan(o.as_strided((count, 5), (o.stride(0), 1), o.storage_offset() + dim)[: count - 1]).all()
    assert int(flags) == (16 if (t >= vocab).any() else 0)


def test_lookup_shapes_and_no_tokens():
    w = torch.randn(50, 12, device="cuda")
    t = torch.randint(0, 50, (2, 3, 4), device="cuda")
    assert torch.equal(_dobb().embedding(w, t), w[t])
    assert _dobb().embedding(w, t[:0]).shape == (0, 3, 4, 12)


def _check_backward(grad, t, vocab, scale, gdt, odt, add, got):
    want, size = L.embedding_backward(grad, t, vocab, scale, add)
    c = np.bincount(t[(t >= 0) & (t < vocab)], minlength=vocab)[:, None]
    bound = (c + 3) * U * size + HALF_UNIT[odt] * np.abs(want) * (1 + 1e-3) + TINY[odt]
    err = np.abs(np64(got) - want)
    assert (err <= bound).all(), float((err - bound).max())
    if add is None:
        assert not np64(got)[c[:, 0] == 0].any()


def _tokens(kind, count, vocab, rng):
    if kind == "uniform":
        return rng.integers(0, vocab, count)
    if kind == "one":                                 # a single token, over and over
        return np.full(count, vocab - 1)
    if kind == "few":                                 # three tokens and padding
        return rng.choice([0, vocab // 2, vocab - 1, -1, -100], count)
    p = 1.0 / (np.arange(vocab) + 2.7)                # frequencies as in text
    return rng.choice(vocab, count, p=p / p.sum())


@pytest.mark.parametrize("gdt", ["f32", "bf16"])
@pytest.mark.parametrize("odt", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["uniform", "one", "few", "text"])
@pytest.mark.parametrize("count,vocab,dim", [(1, 1, 1), (1, 300, 5), (31, 7, 64), (33, 256, 129), (700, 255, 40), (1500, 257, 200),
                                             (5000, 1000, 8)])
def test_gradient(gdt, odt, kind, count, vocab, dim):
    rng = np.random.default_rng(count * 3 + vocab)
    grad = rounded(rng.standard_normal((count, dim)), gdt)
    t = _tokens(kind, count, vocab, rng)
    gd, td = dev(grad, gdt), torch.from_numpy(t).cuda()
    got = _dobb().embedding_backward(gd, td, vocab, scale=1.5, dtype=TORCH[odt])
    _check_backward(grad, t, vocab, 1.5, gdt, odt, None, got)
    # onto what is there; rows of other tokens keep their bits
    old = rounded(rng.standard_normal((vocab, dim)), odt)
    add = dev(old, odt)
    _dobb().embedding_backward(gd, td, scale=1.5, out=add, accumulate=True)
    _check_backward(grad, t, vocab, 1.5, gdt, odt, old, add)
    rest = np.setdiff1d(np.arange(vocab), t)
    assert np.array_equal(np64(add)[rest], old[rest].astype(np.float64))


@pytest.mark.parametrize("gdt,odt", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("dim,extra,offset", [(1601, 0, 0), (63, 1, 1), (1600, 16, 3), (256, 8, 8), (2500, 0, 0)])
def test_gradient_strides_and_offsets(gdt, odt, dim, extra, offset):
    count, vocab = 900, 400
    rng = np.random.default_rng(dim)
    grad = rounded(rng.standard_normal((count, dim)), gdt)
    t = _tokens("text", count, vocab, rng)
    t[::9] = -1
    t[5] = vocab + 3
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = strided(np.ones((vocab, dim)), odt, extra + 2, offset)
    for tdt in (torch.int64, torch.int32):
        out.fill_(7.0)
        td = torch.from_numpy(t).to("cuda", tdt)
        _dobb().embedding_backward(strided(grad, gdt, extra, offset), td, out=out, flags=flags)
        _check_backward(grad, t, vocab, 1.0, gdt, odt, None, out)
        assert torch.isnan(out.as_strided((vocab, extra + 2), (out.stride(0), 1), out.storage_offset() + dim)[: vocab - 1]).all()
    assert int(flags) == 16


@pytest.mark.parametrize("count,vocab,kind", [(40000, 50257, "text"), (70001, 128256, "uniform"), (100000, 70000, "one"),
                                              (8192, 50257, "few"), (262200, 300, "text")])
def test_gradient_of_many_tokens(count, vocab, kind):
    dim = 6
    rng = np.random.default_rng(count)
    grad = rounded(rng.standard_normal((count, dim)), "bf16")
    t = _tokens(kind, count, vocab, rng)
    gd, td = dev(grad, "bf16"), torch.from_numpy(t).cuda()
    got = _dobb().embedding_backward(gd, td, vocab, dtype=torch.float32)
    _check_backward(grad, t, vocab, 1.0, "bf16", "f32", None, got)
    for _ in range(3):     # the order of the sums is fixed: the same bits every time
        assert torch.equal(got, _dobb().embedding_backward(gd, td, vocab, dtype=torch.float32))


@pytest.mark.parametrize("gdt,odt", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32")])
@pytest.mark.parametrize("dim", [5, 512, 1601])
def test_runs_of_every_length(gdt, odt, dim):
    """Tokens that come 1, 2, 3 ... 90 times, then 700 times, in a shuffled
    order: their runs begin at every offset within a unit of the sum and reach
    over any number of units."""
    c = np.concatenate([np.arange(1, 91), [700]])
    rng = np.random.default_rng(dim + 1)
    t = rng.permutation(np.repeat(np.arange(c.size), c))
    grad = rounded(rng.standard_normal((t.size, dim)), gdt)
    gd, td = dev(grad, gdt), torch.from_numpy(t).cuda()
    before = rounded(rng.standard_normal((c.size, dim)), odt)
    for add in (None, before):
        out = dev(before, odt).clone()
        _dobb().embedding_backward(gd, td, out=out, accumulate=add is not None)
        _check_backward(grad, t, c.size, 1.0, gdt, odt, add, out)


def test_gradient_against_differences():
    """<dout, embedding(W)> is linear in W: its difference quotient is exact,
    up to fp32 rounding of the lookups' products (2 u of each of 64 terms)."""
    rng = np.random.default_rng(9)
    w = rng.standard_normal((20, 4)).astype(np.float32)
    t = rng.integers(-1, 20, 64)
    go = rng.standard_normal((64, 4)).astype(np.float32)
    td = torch.from_numpy(t).cuda()
    d = np64(_dobb().embedding_backward(dev(go, "f32"), td, 20, scale=0.5))
    for v in (0, 3, 19):
        for j in range(4):
            up, down = w.copy(), w.copy()
            up[v, j], down[v, j] = 1.0, -1.0
            f = [float((np64(_dobb().embedding(dev(a, "f32"), td, scale=0.5)) * go).sum()) for a in (up, down)]
            assert abs(d[v, j] - (f[0] - f[1]) / 2) <= 64 * 4 * U * np.abs(go).sum()


def test_no_tokens_only_padding_and_a_side_stream():
    d = _dobb()
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    out = torch.full((9, 5), 3.0, device="cuda")
    d.embedding_backward(torch.empty(0, 5, device="cuda"), none, out=out, accumulate=True)
    assert (out == 3.0).all()
    d.embedding_backward(torch.ones(4, 5, device="cuda"), torch.full((4,), -1, device="cuda"), out=out, accumulate=True)
    assert (out == 3.0).all()
    assert not d.embedding_backward(torch.empty(0, 5, device="cuda"), none, out=out).any()
    out.fill_(3.0)
    assert not d.embedding_backward(torch.ones(4, 5, device="cuda"), torch.full((4,), -1, device="cuda"), out=out).any()
    g = torch.randn(3, 50, 24, device="cuda")
    t = torch.randint(0, 99, (3, 50), device="cuda")
    want = d.embedding_backward(g, t, 99)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = d.embedding_backward(g, t, 99, stream=side)
    side.synchronize()
    assert torch.equal(got, want)


def test_rows_past_32_bit_offsets():
    vocab, dim, stride = 5, 40, (1 << 29) + 9
    buf = torch.zeros((vocab - 1) * stride + dim, dtype=torch.bfloat16, device="cuda")
    w = torch.as_strided(buf, (vocab, dim), (stride, 1))
    src = torch.randn(vocab, dim, device="cuda").bfloat16()
    w.copy_(src)
    t = torch.tensor([4, 0, 4, 3], device="cuda")
    assert torch.equal(_dobb().embedding(w, t), src[t])
    g = torch.randn(4, dim, device="cuda")
    want = _dobb().embedding_backward(g, t, vocab, dtype=torch.bfloat16)
    _dobb().embedding_backward(g, t, out=w)
    assert torch.equal(w, want)
