"""Sampling at the ends of the numbers: logits whose differences leave fp32, and what else lies there.
The bounds are those of test_gpu_lm_sample."""
import numpy as np
import pytest

from lm_util import dev, rounded
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


@pytest.mark.parametrize("xt", ["f32", "bf16"])
def test_a_random_number_of_zero_wins_with_the_lowest_logit_too(xt):
    """scale * (logit - max) beyond fp32 next to -log 0: by the list, by the whole row and the general way."""
    import block_eigenbasis_preconditioning_gb300 as d
    rng = np.random.default_rng(22)
    low = rounded(np.array([-3.38e38]), xt)[0]
    for vocab in (600, 20000):
        x = np.full((5, vocab), -np.inf, dtype=np.float32)
        x[:, :50] = rounded(rng.normal(size=(5, 50)), xt)
        x[:, 100:110] = low
        e = rounded(rng.exponential(size=x.shape), "f32")
        e[:, 105], e[1, 105], e[2, 107] = 0.0, -0.0, 0.0
        e[4, 200] = 0.0  # of a token that cannot occur: not looked at
        for scale, top_k in ((2.0, 0), (2.0, 58), (1e6, 0), (1e6, 58), (2.0 ** 127, 58)):
            r = d.sample(dev(x, xt), dev(e, "f32"), scale=scale, top_k=top_k)
            assert r.tokens.tolist() == [105] * 5 and bool((r.logp == -np.inf).all()), (vocab, scale, top_k)
            # among fewer the zero is not kept
            assert bool((d.sample(dev(x, xt), dev(e, "f32"), scale=scale, top_k=55).tokens < 50).all())
