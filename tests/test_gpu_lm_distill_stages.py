"""Distillation's loss and gradient where rows of one block differ by a vector at a stage's border, so that the
last entries of one lie where the next one's copy goes.

Against fp64 on the device: with w_j = scale (x_j - max), an entry p_j of the gradient is off by
(4 |w_j| + 2 W + 3 |log sum| + chain + 40) u of itself (lm_util; W = sum p |w|), the teacher's
q_i by (4 |w_i| + 2 W_t + 2 |log sum_t| + 60) u: bounded by the largest |w| of a row."""
import pytest
import torch

from lm_util import U, chain

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,rows,vocab,gap", [
    (torch.float32, 257, 147500, 1), (torch.float32, 257, 147500, 3), (torch.float32, 257, 147501, 0),  # 24580 = 3 stages and a vector in the last block
    (torch.bfloat16, 110, 294960, 1), (torch.bfloat16, 110, 294960, 5),                                  # 49160 in each of six
    (torch.bfloat16, 512, 98320, 1), (torch.bfloat16, 512, 98320, 0),                                    # 49160 in each of two
    (torch.float32, 330, 8196, 1), (torch.bfloat16, 330, 16392, 1), (torch.float32, 400, 3, 0), (torch.bfloat16, 700, 9, 2)])
def test_a_vector_more_or_less_at_the_border_of_a_stage(dtype, rows, vocab, gap):
    import block_eigenbasis_preconditioning_gb300 as d
    g = torch.Generator("cuda").manual_seed(vocab + gap)
    x = (2.0 * torch.randn(rows, vocab + gap, device="cuda", generator=g)).to(dtype)[:, :vocab]
    x[:, -8:] += 8.0  # what stands behind the vectors weighs
    k = min(vocab, 12)
    ids = torch.rand(rows, min(vocab, 4096), device="cuda", generator=g).topk(k).indices.int()
    t, gl = torch.randn(rows, k, device="cuda", generator=g), 0.5 + torch.rand(rows, device="cuda", generator=g)
    r = d.distill(x, ids, t, grad_loss=gl)
    q = torch.softmax(t.double(), 1)
    for lo in range(0, rows, 64):
        at = slice(lo, lo + 64)
        logp = torch.log_softmax(x[at].double(), 1)
        rel = U * (8 * float((x[at].amax(1) - x[at].amin(1)).max()) + 4 * float(-logp.max()) + 64 + chain(vocab) + 60)
        want = logp.exp()
        size = want.scatter_add(1, ids[at].long(), q[at])
        want = gl[at, None].double() * want.scatter_add(1, ids[at].long(), -q[at])
        bound = gl[at, None].double() * size * rel
        if dtype == torch.bfloat16:
            bound += 2.0 ** -8 * (want.abs() + bound)
        assert bool(((r.grad[at].double() - want).abs() <= bound + 1e-44).all())
        loss = (torch.special.xlogy(q[at], q[at]) - q[at] * logp.gather(1, ids[at].long())).sum(1)
        assert bool(((r.loss[at].double() - loss).abs() <= rel * (1 + loss.abs() + logp.gather(1, ids[at].long()).abs().amax(1))).all())
    again = d.distill(x, ids, t, grad_loss=gl)
    assert torch.equal(again.grad, r.grad) and torch.equal(again.loss, r.loss)
    y = x.clone(memory_format=torch.preserve_format) if gap == 0 else torch.empty(rows, vocab + gap, dtype=dtype, device="cuda")[:, :vocab].copy_(x)
    assert torch.equal(d.distill(y, ids, t, grad_loss=gl, out=y).grad, r.grad)
