"""Layer norm of finite rows whose factors leave fp32: the results are finite."""
import numpy as np
import pytest
import torch

from lm_util import U, assert_close, dev, np64, rounded

pytestmark = pytest.mark.gpu
C = 48  # as in test_gpu_lm_norm


@pytest.mark.parametrize("xt", ["f32", "bf16"])
@pytest.mark.parametrize("dim", [16, 64, 1024, 4096, 16384, 32768])
def test_a_gain_that_is_too_large_for_the_rows_factor(dim, xt):
    """rstd weight beyond fp32, their product with the row's differences not."""
    import block_eigenbasis_preconditioning_gb300 as d
    x = np.full((9, dim), 3.0, dtype=np.float32)
    bias = rounded(np.random.default_rng(31).normal(size=dim), "f32")
    w = np.full(dim, 1e24, dtype=np.float32)
    r = d.layer_norm(dev(x, xt), dev(w, "f32"), dev(bias, "f32"), eps=1e-30, out_dtype=torch.float32)
    assert np.array_equal(np64(r.out), np.broadcast_to(bias.astype(np.float64), x.shape))


@pytest.mark.parametrize("xt", ["f32", "bf16"])
@pytest.mark.parametrize("eps", [1e-20, 2.0 ** -126])
@pytest.mark.parametrize("dim", [16, 64, 1024, 4096, 16384, 32768])
def test_constant_rows_of_large_numbers(dim, xt, eps):
    """Powers of two wide, numbers of few bits: mean and variance are exact, so xh is 0.  dx = rstd (g - mean g), off
    by the roundings of mean(g) (C + 4), of rstd (4) and of the expression (6), as test_gpu_lm_norm has them."""
    import block_eigenbasis_preconditioning_gb300 as d
    rng = np.random.default_rng(32)
    x = np.repeat(np.array([1.75 * 2.0 ** 127, -1.75 * 2.0 ** 127, 1.5 * 2.0 ** 104, -1.5 * 2.0 ** 100, 2.5, 0.0], dtype=np.float32)[:, None], dim, 1)
    bias, g = rounded(rng.normal(size=dim), "f32"), rounded(rng.normal(size=x.shape), "f32")
    xd = dev(x, xt)
    r = d.layer_norm(xd, None, dev(bias, "f32"), eps=eps, out_dtype=torch.float32)
    rstd = 1.0 / np.sqrt(float(np.float32(eps)))
    assert np.array_equal(np64(r.mean), x[:, 0].astype(np.float64))
    assert np.abs(np64(r.rstd) / rstd - 1).max() < 4 * U
    assert np.array_equal(np64(r.out), np.broadcast_to(bias.astype(np.float64), x.shape))
    q = d.layer_norm_backward(dev(g, "f32"), xd, r)
    g = g.astype(np.float64)
    m1, size = g.mean(1, keepdims=True), np.abs(g).mean(1, keepdims=True)
    want = rstd * (g - m1)
    bound = rstd * U * ((C + 4) * size + 10 * (np.abs(g) + size))
    assert_close(np64(q.x), want, bound + (0 if xt == "f32" else 2.0 ** -8 * (np.abs(want) + bound)), "dx")
    assert not q.weight.any()
    assert_close(np64(q.bias), g.sum(0), (len(x) + 64) * U * np.abs(g).sum(0), "dbias")
