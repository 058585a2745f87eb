"""Distillation from entries whose log probability leaves fp32 although their share of the loss does not.  The
bounds are those of test_gpu_lm_distill; a power below 2^-126 is 0, so that p_j is off by that much more, the gradient by
2^-126 scale |g|."""
import numpy as np
import pytest
import torch

from lm_util import HALF_UNIT, TINY, U, assert_close, dev, np64, rounded
from oracle import lm as O
from test_gpu_lm_distill import _bounds, _inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("xt", ["f32", "bf16"])
@pytest.mark.parametrize("rows,vocab", [(6, 700), (400, 3000), (4, 60000)])
def test_masks_of_the_lowest_value_under_a_large_scale(xt, rows, vocab):
    x, ids, t, g = _inputs(rows, vocab, 7, xt, "f32", 71)
    low = float(rounded(np.array([-3.38e38]), xt)[0])
    x[np.arange(rows), ids[:, 2]] = low
    x[0, ids[0, 4]] = low
    t[:, 2] -= 2.0  # a share of the loss that fp32 holds
    t[1, 2] += 30.0  # all of it: beyond fp32
    t[2, 2] = -np.inf
    x[3, ids[3, 2]] = -np.inf
    import block_eigenbasis_preconditioning_gb300 as d
    xd, idd, td, gd = dev(x, xt), torch.from_numpy(ids).cuda(), dev(t, "f32"), dev(g, "f32")
    for scale, ts in ((1.5, 1.0), (2.0, 1.0), (20.0, 1.5)):
        loss, dl = O.distill(x, ids, t, scale, ts), O.distill_backward(x, ids, t, g, scale, ts)
        el, eg = _bounds(x, ids, t, g, scale, ts, xt)
        eg = eg + (2.0 ** -126 * scale * np.abs(g))[:, None]
        eg = eg + HALF_UNIT[xt] * (np.abs(dl) + eg) + 4 * TINY[xt]
        el = el + U * np.where(np.isfinite(loss), np.abs(loss), 0) + 1e-45
        f, both = d.distill(xd, idd, td, scale=scale, teacher_scale=ts), d.distill(xd, idd, td, scale=scale, teacher_scale=ts, grad_loss=gd)
        for what, r in (("loss", f), ("loss with gradient", both)):
            assert_close(np64(r.loss), loss, el, what)
        for what, grad in (("gradient", d.distill_backward(xd, idd, td, f, gd)), ("gradient with loss", both.grad)):
            assert_close(np64(grad), dl, eg, what)
        assert np.isfinite(loss[0]) and loss[0] > 1e30 and np.abs(loss[1]) > 3e38 and loss[3] == np.inf
