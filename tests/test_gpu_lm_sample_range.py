"""Sampling at the ends of the numbers: logits whose differences leave fp32, and what else lies there.
The bounds are those of test_gpu_lm_sample."""
import numpy as np
import pytest

from lm_util import rounded
from test_gpu_lm_sample import _check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("xt", ["f32", "bf16"])
@pytest.mark.parametrize("rows,vocab", [(6, 900), (2, 40001)])
def test_logits_whose_differences_leave_fp32(xt, rows, vocab):
    """Logits up to the ends of fp32 under a scale that makes ordinary numbers of them."""
    rng = np.random.default_rng(21)
    x = rounded(rng.uniform(-3.3e38, 3.3e38, size=(rows, vocab)), xt)
    x[0, :4] = rounded(np.array([3.3e38, 0.0, 0.0, -3.3e38]), xt)
    x[0, 4:] = -np.inf
    e = rounded(rng.exponential(size=x.shape), "f32")
    e[0, 3] = 1e-6  # the lowest one wins where it is kept
    for f in (dict(), dict(min_p=1e-4), dict(top_p=0.9999), dict(top_p=0.6), dict(top_k=4), dict(top_k=700), dict(top_k=500, top_p=0.9, min_p=1e-4)):
        r = _check(x, e, xt, scale=2.0 ** -126, **f)
        assert int(r.tokens[0]) == (0 if f.get("top_p", 1.0) <= 0.9 else 3)  # (the first has 0.96 of the mass)
