"""Log probabilities of logits near both ends of fp32 at a scale that brings
them back to ordinary numbers: the difference of two logits exceeds fp32, its
product with the scale does not (bounds: lm_util; probabilities below 2^-126
count as 0, as the exponential says, so what they bring may be lost)."""
import numpy as np
import pytest
import torch

from oracle import lm as L

from lm_util import HALF_UNIT, TINY, assert_close, grad_bound, np64, rounded
from test_gpu_lm_logprobs import _check_forward, _dobb, _forward

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,vocab", [(1, 7), (3, 2051), (2, 40001), (640, 511), (640, 4999), (310, 17003)])
@pytest.mark.parametrize("scale", [2.0 ** -126, 2.0 ** -122, 0.5])
def test_differences_beyond_fp32(dtype, rows, vocab, scale):
    rng = np.random.default_rng(vocab)
    x = rounded(rng.uniform(-3.3e38, 3.3e38, (rows, vocab)), dtype)
    x[0, 0] = -np.inf
    x[rows // 2, 1:3] = rounded(np.array([3.3e38, -3.3e38]), dtype)
    t = rng.integers(0, vocab, rows)
    t[rows // 2] = 2
    k = 5
    xd, td, r = _forward(x, t, dtype, scale, k)
    f, eS, eH = _check_forward(x, t, r, scale, k)
    g, h = (rng.standard_normal(rows).astype(np.float32) for _ in range(2))
    cu = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    big = np.float32(2.0 ** 100)             # so that the gradients are ordinary numbers, too
    d = np64(_dobb().log_probs_backward(xd, td, r, cu(g * big), grad_entropy=cu(h * big)))
    want = L.log_probs_backward(x, t, g * big, h * big, None, scale)
    b = grad_bound(x, t, f, eS, eH, g * big, h * big, None, scale, dtype)
    lp = scale * (x.astype(np.float64) - f["row_max"][:, None]) - f["log_sum"][:, None]
    with np.errstate(invalid="ignore"):
        size = np.abs(g * big)[:, None] + np.abs(h * big)[:, None] * (np.abs(lp) + f["entropy"][:, None])
        b += np.where((lp < -125 * np.log(2.0)) & np.isfinite(lp), scale * np.exp(lp) * size, 0.0)
    assert_close(d, want, b + HALF_UNIT[dtype] * np.abs(want) * (1 + 1e-3) + TINY[dtype], "dlogits")
