"""Layer norm of finite rows whose factors leave fp32: the results are finite."""
import numpy as np
import pytest
import torch

from lm_util import dev, np64, rounded

pytestmark = pytest.mark.gpu


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
