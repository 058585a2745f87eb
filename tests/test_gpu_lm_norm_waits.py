"""Rows of layer norm that a wait gave up on: copies that are never made, bounded waits that run out and NaN;
the rows before are whole, and so is the next call."""
import time

import pytest
import torch

pytestmark = pytest.mark.gpu
CODES = {torch.float32: 0, torch.bfloat16: 1}
SIZES = [(torch.bfloat16, 3000, 1600), (torch.float32, 2000, 4096), (torch.float32, 700, 10000), (torch.float32, 900, 1601), (torch.bfloat16, 100, 5000)]


def _data(dtype, rows, dim):
    g = torch.Generator("cuda").manual_seed(rows)
    randn = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    return randn(rows, dim).to(dtype), randn(rows, dim).to(dtype), 1.0 + 0.2 * randn(dim)


def _stream():
    return torch.cuda.current_stream().cuda_stream


def _forward(x, w, loaded, limit_ns):
    from block_eigenbasis_preconditioning_gb300 import binding
    (rows, dim), t = x.shape, CODES[x.dtype]
    out, stats = torch.full_like(x, 7.0), torch.full((2, rows), 7.0, device="cuda")
    st = binding.load_library().dobb_selftest_layer_norm_timeout(
        x.data_ptr(), t, rows, dim, dim, w.data_ptr(), None, 0, 1e-5, out.data_ptr(), t, dim, stats[0].data_ptr(), stats[1].data_ptr(), _stream(),
        loaded, limit_ns)
    return st, out, stats


def _backward(g, x, r, w, loaded, limit_ns):
    from block_eigenbasis_preconditioning_gb300 import binding
    (rows, dim), t, lib = x.shape, CODES[x.dtype], binding.load_library()
    dx, dp = torch.full_like(x, 7.0), torch.full((2, dim), 7.0, device="cuda")
    ws = torch.empty(lib.dobb_layer_norm_backward_bytes(rows, dim), dtype=torch.uint8, device="cuda")
    st = lib.dobb_selftest_layer_norm_backward_timeout(
        g.data_ptr(), t, dim, x.data_ptr(), t, rows, dim, dim, w.data_ptr(), 0, r.mean.data_ptr(), r.rstd.data_ptr(), dx.data_ptr(), dim,
        dp[0].data_ptr(), dp[1].data_ptr(), 0, 0, ws.data_ptr(), ws.numel(), _stream(), loaded, limit_ns)
    return st, dx, dp


@pytest.mark.parametrize("dtype,rows,dim", SIZES)
@pytest.mark.parametrize("share", [0.0, 0.4, 1.0])
def test_lost_rows_are_nan(dtype, rows, dim, share):
    import block_eigenbasis_preconditioning_gb300 as d
    x, g, w = _data(dtype, rows, dim)
    loaded = int(rows * share)
    want = d.layer_norm(x, w)
    grads = d.layer_norm_backward(g, x, want, w)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    st, out, stats = _forward(x, w, loaded, 50_000_000)
    assert st == 0
    st, dx, dp = _backward(g, x, want, w, loaded, 50_000_000)
    assert st == 0
    torch.cuda.synchronize()
    assert time.perf_counter() - t0 < 5.0
    for got, whole in ((out, want.out), (stats[0], want.mean), (stats[1], want.rstd)):
        assert torch.equal(got[:loaded], whole[:loaded]) and bool(got[loaded:].isnan().all())
    # (a copy of the gradients has up to fifteen rows)
    assert torch.equal(dx[:loaded], grads.x[:loaded]) and bool(dx[loaded + 15:].isnan().all())
    if share == 1.0:
        assert torch.equal(dp[0], grads.weight) and torch.equal(dp[1], grads.bias)
    else:
        assert bool(dp.isnan().all())
    again = d.layer_norm(x, w)
    back = d.layer_norm_backward(g, x, again, w)
    assert torch.equal(again.out, want.out) and all(torch.equal(a, b) for a, b in zip(back, grads))


def test_limits_of_the_self_tests():
    import block_eigenbasis_preconditioning_gb300 as d
    x, g, w = _data(torch.float32, 40, 512)
    r = d.layer_norm(x, w)
    for loaded, limit in ((41, 10 ** 6), (-1, 10 ** 6), (4, 0), (4, 6 * 10 ** 9)):
        (st, out, stats), (sb, dx, dp) = _forward(x, w, loaded, limit), _backward(g, x, r, w, loaded, limit)
        torch.cuda.synchronize()
        assert st == sb == 1 and all(bool((t == 7.0).all()) for t in (out, stats, dx, dp))
    x, g, w = _data(torch.float32, 3, 20000)
    assert _forward(x, w, 1, 10 ** 6)[0] == 6 and _backward(g, x, d.layer_norm(x, w), w, 1, 10 ** 6)[0] == 6
