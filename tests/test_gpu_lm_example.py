"""The operators together, as the example uses them: the gradients of the whole
model against fp64 autograd, and a short training run."""
import math
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def test_model_gradients_against_fp64_autograd():
    """fp32 weights: every product is a sum of at most 300 terms and there are
    four in a row, so 4 (300 + 60) u of the largest value bounds the error
    (u = 2^-24; TF32 off)."""
    import tied_lm as ex
    gen = torch.Generator(device="cuda").manual_seed(1)
    vocab, dim, n = 300, 64, 200
    E = torch.randn(vocab, dim, device="cuda", generator=gen) * 0.05
    W = torch.randn(dim, dim, device="cuda", generator=gen) / math.sqrt(dim)
    cur, nxt = ex.batch(n, vocab, gen)
    assert not torch.backends.cuda.matmul.allow_tf32
    loss, dE, dW, _, _ = ex.loss_and_gradients(E, W, cur, nxt)
    e, w = E.double().requires_grad_(), W.double().requires_grad_()
    logp = torch.log_softmax((e[cur] * math.sqrt(dim)) @ w.t() @ e.t(), 1)
    want = -logp.gather(1, nxt[:, None]).mean() + ex.ENTROPY_WEIGHT * (logp.exp() * logp).sum(1).mean()
    want.backward()
    bound = 4 * 360 * 2.0 ** -24
    assert abs(float(loss) - want.item()) <= bound * abs(want.item())
    for got, ref in ((dE, e.grad), (dW, w.grad)):
        assert float((got.double() - ref).abs().max()) <= bound * float(ref.abs().max())


def test_example_learns_the_walk():
    """Four fifths of the steps of the walk can be known: the loss has to come
    down from log(vocab) by a nat at least, and the likeliest next token is the
    walk's for most tokens."""
    import tied_lm as ex
    losses, norms, (E, W) = ex.train(steps=60)
    assert abs(losses[0] - math.log(1000)) < 0.5
    assert losses[-1] < losses[0] - 1.0 and all(math.isfinite(v) for v in losses + norms)
    right = sum(ex.continue_from(E, W, t)[0][0] == (7 * t + 3) % 1000 for t in range(0, 1000, 25))
    assert right >= 20
