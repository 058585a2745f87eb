"""Sampling at the ends of the numbers: logits whose differences leave fp32, and what else lies there.
The bounds are those of test_gpu_lm_sample."""
import numpy as np
import pytest
import torch

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


def test_top_p_over_half_a_million_nearly_equal_masses():
    """One block a row, three quarters of it one value whose sum rounds one way again and again (a plain
    fp32 sum is off by up to 2^-17 of itself): what is kept is right to (3 W + 32) u of the mass, W the mean |log| of a
    mass, u = 2^-24, as dobb.h has it.

    Around the border the random numbers are tiny, the smaller the further behind: the token names the last entry kept."""
    import block_eigenbasis_preconditioning_gb300 as d
    rows, vocab, first, around = 312, 524288, 1024, 12
    rng = np.random.default_rng(23)
    behind = np.linspace(0.21, 0.9, 12)  # of the one value, in units of log 2
    x = np.zeros((len(behind), vocab), dtype=np.float32)  # (the maximum first: nothing is moved later)
    x[:, first:first + vocab * 3 // 4] = -np.log(2) * behind[:, None]
    x[:, first + vocab * 3 // 4:] = rng.uniform(-3 * np.log(2), -np.log(2), size=(len(behind), vocab - first - vocab * 3 // 4))  # few near each border
    order = np.argsort(-x, axis=1, kind="stable")
    p = np.exp(np.take_along_axis(x, order, 1).astype(np.float64))
    total, upto = p.sum(1), p.cumsum(1)
    slack = (3 * (p * -np.log(p)).sum(1) / total + 32) * 2.0 ** -24 * total
    which = np.arange(rows) % len(behind)
    top_p = rng.uniform(0.92, 0.98, size=rows).astype(np.float32)
    share = top_p.astype(np.float64) * total[which]
    last = np.array([int(np.searchsorted(upto[r], s)) for r, s in zip(which, share)])  # before it lies less
    noise = torch.ones(rows, vocab, device="cuda")
    at = np.stack([order[r, n - around:n + around] for r, n in zip(which, last)])
    noise.scatter_(1, torch.from_numpy(at).cuda(), torch.logspace(-3, -36, 2 * around, device="cuda").expand(rows, -1))
    r = d.sample(torch.from_numpy(x).cuda()[torch.from_numpy(which).cuda()], noise, top_p=torch.from_numpy(top_p).cuda())
    rank = np.argsort(order, axis=1)
    kept = rank[which, r.tokens.cpu().numpy()]
    off = np.maximum(upto[which, kept - 1] - share, share - upto[which, kept]) / slack[which]
    assert (off <= 1).all(), f"{int((off > 1).sum())} of {rows} rows end {off.max():.1f} times too far from the border ({kept[off.argmax()] - last[off.argmax()]} entries)"


@pytest.mark.parametrize("offset", [40000.0, -37000.0, 700.0])
def test_min_p_that_ends_right_behind_top_p(offset):
    """Logits far from 0, so that what top_p's bins are relative to is coarse in fp32 (2^-9 of a power of two), and
    a gap below the border: min_p ends in the gap, top_p a few entries before it."""
    import block_eigenbasis_preconditioning_gb300 as d
    rows, vocab, upper, around = 256, 40000, 20000, 40
    rng = np.random.default_rng(24)
    x = np.empty((rows, vocab), dtype=np.float32)
    x[:, :upper] = offset + rng.uniform(-0.2, 0, size=(rows, upper))
    x[:, upper:] = offset + rng.uniform(-3.2, -3, size=(rows, vocab - upper))
    order = np.argsort(-x, axis=1, kind="stable")
    s = np.take_along_axis(x, order, 1).astype(np.float64)
    p = np.exp(s - s[:, :1])
    upto = p.cumsum(1)
    top_p = np.float32(upto[:, upper - 1] / upto[:, -1] - np.linspace(2e-5, 1.5e-3, rows))
    share = top_p.astype(np.float64) * upto[:, -1]
    last = (upto < share[:, None]).sum(1)  # the entry that crosses the border is kept
    noise = torch.ones(rows, vocab, device="cuda")
    at = np.stack([order[i, upper - 2 * around:upper] for i in range(rows)])
    noise.scatter_(1, torch.from_numpy(at).cuda(), torch.logspace(-2, -36, 2 * around, device="cuda").expand(rows, -1))
    r = d.sample(torch.from_numpy(x).cuda(), noise, top_p=torch.from_numpy(top_p).cuda(), min_p=float(np.exp(-1.5)))
    kept = np.array([int(np.where(order[i] == int(t))[0][0]) for i, t in enumerate(r.tokens.cpu())])
    w = (p * -np.log(p)).sum(1) / upto[:, -1]
    slack = (3 * w + 32) * 2.0 ** -24 * upto[:, -1]
    i = np.arange(rows)
    off = np.maximum(np.where(kept > 0, upto[i, kept - 1], 0.0) - share, share - upto[i, kept]) / slack
    assert (off <= 1).all(), f"{int((off > 1).sum())} of {rows} rows, up to {(kept - last)[off.argmax()]} entries off"
