"""Outputs that share memory with what the same call reads or writes elsewhere
are refused before any device work (made-up addresses, no GPU)."""
import ctypes

import pytest
import torch

from block_eigenbasis_preconditioning_gb300 import binding

P = 1 << 20        # a made-up device address
FREE = 1 << 40     # another, far from all others


@pytest.fixture(scope="module")
def lib():
    if torch.cuda.is_available():
        pytest.skip("a call that is not refused would run on made-up addresses")
    return binding.load_library()


def _refused(lib, st):
    return st == 1 and b"overlap" in lib.dobb_last_error()


def _clip(lib, g, gd, ne, out, od):
    ptr = lambda v: (ctypes.c_void_p * len(v))(*v)  # noqa: E731
    i32 = lambda v: (ctypes.c_int32 * len(v))(*v)  # noqa: E731
    st = lib.dobb_clip_grads(len(g), ptr(g), i32(gd), (ctypes.c_int64 * len(ne))(*ne), 1.0, None if out is None else ptr(out),
                             None if out is None else i32(od), FREE, None, FREE + (1 << 20), 1 << 20, None)
    return _refused(lib, st)


@pytest.mark.parametrize("g,gd,ne,out,od,refused", [
    ((P, P), (0, 0), (16, 16), (P, P), (0, 0), True),                                  # a tied gradient, listed twice
    ((P, P + 64), (0, 0), (16, 16), (P, P + 64), (0, 0), False),                       # neighbours, in place
    ((P, P + 60), (0, 0), (16, 16), (P, P + 60), (0, 0), True),
    ((P + 32, P), (1, 1), (16, 16), (P + 32, P), (1, 1), False),
    ((P + 30, P), (1, 1), (16, 16), (P + 30, P), (1, 1), True),
    ((P, P), (0, 0), (16, 16), (2 * P, 3 * P), (0, 0), False),                         # read twice
    ((P, P), (0, 0), (16, 16), (P, 3 * P), (0, 0), True),                              # read by one, written by the other
    ((P, 2 * P), (0, 0), (16, 16), (3 * P, 3 * P), (0, 0), True),                      # two outputs on one place
    ((P, 2 * P), (0, 0), (16, 16), (2 * P, P), (0, 0), True),                          # exchanged
    ((P, 2 * P), (0, 0), (16, 16), (P + 4, 3 * P), (0, 0), True),                      # over its own gradient, shifted
    ((P, 2 * P), (0, 0), (16, 16), (P + 64, 3 * P), (1, 1), False),
    ((P, 2 * P), (0, 1), (16, 16), (P + 60, 3 * P), (1, 1), True),
    ((P, P, P + 8), (0, 0, 0), (16, 0, 0), (P, P, P + 4), (0, 0, 0), False),           # empty ones are nowhere
    ((P, P + 4096, P + 64), (0, 0, 0), (1 << 20, 1, 1), (P, FREE, FREE + 8), (0, 0, 0), True),    # within a long one
    ((P, P + 4096, 2 * P), (0, 0, 0), (16, 1 << 20, 4), (P, P + 4096, 2 * P), (0, 0, 0), True),
    ((P, P), (0, 0), (16, 16), None, None, False)])                                    # norms only
def test_clip(lib, g, gd, ne, out, od, refused):
    assert _clip(lib, g, gd, ne, out, od) is refused


def test_clip_of_many_tensors_in_any_order(lib):
    gen = torch.Generator().manual_seed(1)
    for n in (700, 40):
        order = torch.randperm(n, generator=gen).tolist()
        g = [P + 64 * i for i in order]
        assert not _clip(lib, g, [0] * n, [16] * n, g, [0] * n)
        assert not _clip(lib, g, [0] * n, [16] * n, [FREE + (1 << 30) + 32 * i for i in order], [1] * n)
        bad = list(g)
        bad[n // 2] = bad[n // 3]
        assert _clip(lib, bad, [0] * n, [16] * n, bad, [0] * n)
        assert _clip(lib, g, [0] * n, [16] * (n - 1) + [17 if order[-1] < n - 1 else 16], g, [0] * n) is (order[-1] < n - 1)


@pytest.mark.gpu
def test_a_gradient_listed_twice_is_refused():
    import block_eigenbasis_preconditioning_gb300 as d
    x, y = torch.ones(1000, device="cuda"), torch.ones(70, device="cuda")
    for call in (lambda: d.clip_grads([x, y, x], 1.0), lambda: d.clip_grads([x[:600], x[500:]], 1.0),
                 lambda: d.clip_grads([x, y], 1.0, out=[torch.empty_like(x), x[5:75]])):
        with pytest.raises(binding.DobbError, match="overlap"):
            call()
    assert bool((x == 1).all())
    assert abs(float(d.grad_norm([x, y, x]).norm) - 2070 ** 0.5) < 1e-4
    d.clip_grads([x[:500], x[500:], y], 1.0)
    assert abs(float(x.double().square().sum() + y.double().square().sum()) - 1.0) < 1e-5


def _rows(at, rows, width, stride):
    """The bytes of a matrix: the definition that the closed form is compared with."""
    return {at + r * stride + c for r in range(rows) for c in range(width)}


def _pairs(seed, count):
    """Small matrices near each other: offset, rows, columns and strides, in elements."""
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda lo, hi: int(torch.randint(lo, hi + 1, (1,), generator=gen))  # noqa: E731
    for _ in range(count):
        cols = rnd(1, 6)
        a, b = (cols + rnd(0, 9) for _ in range(2))
        yield rnd(-60, 60), rnd(1, 7), rnd(1, 7), cols, a, a if rnd(0, 1) else b


def _log_probs_backward(lib, at, rows, vocab, stride, ostride, dtype):
    st = lib.dobb_log_probs_backward(P, dtype, rows, vocab, stride, FREE, 8, 1.0, FREE, FREE, None, FREE, None, None, at, ostride, None)
    return _refused(lib, st)


@pytest.mark.parametrize("dtype", [0, 1])
def test_gradient_of_log_probabilities(lib, dtype):
    b = 2 if dtype else 4
    assert not _log_probs_backward(lib, P, 5, 8, 8, 8, dtype)               # in place
    assert _log_probs_backward(lib, P + 8 * b, 5, 8, 8, 8, dtype)           # a row behind
    assert not _log_probs_backward(lib, P + 40 * b, 5, 8, 8, 8, dtype)
    assert not _log_probs_backward(lib, P + 8 * b, 8192, 8, 16, 16, dtype)  # halves of the same rows
    assert _log_probs_backward(lib, P + 7 * b, 8192, 8, 16, 16, dtype) and _log_probs_backward(lib, P + 9 * b, 8192, 8, 16, 16, dtype)
    assert _log_probs_backward(lib, P - 8000 * 16 * b, 8192, 8, 16, 16, dtype)
    hits = 0
    for off, rows, _, cols, s, t in _pairs(dtype, 3000):
        if off == 0:
            continue
        want = bool(_rows(0, rows, cols, s) & _rows(off, rows, cols, t))
        hits += want
        assert _log_probs_backward(lib, P + off * b, rows, cols, s, t, dtype) is want, (off, rows, cols, s, t)
    assert 300 < hits < 2700


@pytest.mark.gpu
def test_a_gradient_over_part_of_the_logits_is_refused():
    import block_eigenbasis_preconditioning_gb300 as d
    buf = torch.randn(70, 200, device="cuda")
    t, g = torch.zeros(64, dtype=torch.int64, device="cuda"), torch.ones(64, device="cuda")
    x = buf[:64, :100]
    r = d.log_probs(x, t)
    want, kept = d.log_probs_backward(x, t, r, g), x.clone()
    for out in (buf[1:65, :100], buf[:64, 1:101], buf[3:67, 99:199]):
        with pytest.raises(binding.DobbError, match="overlap"):
            d.log_probs_backward(x, t, r, g, out=out)
    assert torch.equal(x, kept)
    assert torch.equal(d.log_probs_backward(x, t, r, g, out=buf[:64, 100:]), want) and torch.equal(x, kept)
    assert torch.equal(d.log_probs_backward(x, t, r, g, out=x), want)


def _check_matrices(call, dtype, seed):
    """call(offset, rows there, rows at P, cols, stride there, stride at P) against the bytes."""
    b, hits = 2 if dtype else 4, 0
    for off, m, n, cols, s, t in _pairs(seed, 3000):
        want = bool(_rows(off, m, cols, s) & _rows(0, n, cols, t))
        hits += want
        assert call(P + off * b, m, n, cols, s, t) is want, (off, m, n, cols, s, t)
    assert 300 < hits < 2700


@pytest.mark.parametrize("dtype", [0, 1])
def test_lookup(lib, dtype):
    def call(at, count, vocab, dim, ostride, wstride):
        return _refused(lib, lib.dobb_embedding(P, dtype, vocab, dim, wstride, FREE, 8, count, 1.0, at, dtype, ostride, None, None))
    _check_matrices(call, dtype, 10 + dtype)
    # 32-bit weights, 16-bit outputs
    mixed = lambda at: _refused(lib, lib.dobb_embedding(P, 0, 100, 8, 8, FREE, 8, 4, 1.0, at, 1, 8, None, None))  # noqa: E731
    assert mixed(P) and mixed(P + 3198) and not mixed(P + 3200) and mixed(P - 62) and not mixed(P - 64)


@pytest.mark.gpu
def test_a_lookup_into_the_weight_is_refused():
    import block_eigenbasis_preconditioning_gb300 as d
    w = torch.randn(50, 64, device="cuda")
    t, kept = torch.arange(20, device="cuda"), w.clone()
    for out in (w[:20], w[30:], w.view(100, 32)[:40].view(20, 64)):
        with pytest.raises(binding.DobbError, match="overlap"):
            d.embedding(w, t, out=out)
    assert torch.equal(w, kept) and torch.equal(d.embedding(w[:30], t, out=w[30:]), kept[:20])


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("accumulate", [0, 1])
def test_gradient_of_the_lookup(lib, dtype, accumulate):
    def call(at, vocab, count, dim, ostride, gstride):
        return _refused(lib, lib.dobb_embedding_backward(P, dtype, count, dim, gstride, FREE, 8, vocab, 1.0, at, dtype, ostride,
                                                         accumulate, None, FREE + (1 << 20), 1 << 30, None))
    _check_matrices(call, dtype, 20 + dtype)


@pytest.mark.gpu
def test_a_gradient_into_itself_is_refused():
    import block_eigenbasis_preconditioning_gb300 as d
    g = torch.randn(50, 64, device="cuda")
    t, kept = torch.arange(20, device="cuda"), g.clone()
    for out in (g[:20], g[19:], g.view(100, 32)[9:39].view(15, 64)):
        for add in (False, True):
            with pytest.raises(binding.DobbError, match="overlap"):
                d.embedding_backward(g[:20], t, out=out, accumulate=add)
    assert torch.equal(g, kept)
    assert torch.equal(d.embedding_backward(g[:20], t, out=g[20:]), torch.cat([kept[:20], torch.zeros(10, 64, device="cuda")]))
