"""Log probabilities, entropies, alternatives and their gradient on the GPU
against the fp64 definitions (bounds: lm_util)."""
import numpy as np
import pytest
import torch

from oracle import lm as L

from lm_util import (HALF_UNIT, TINY, TORCH, U, assert_close, grad_bound, logp_bound, np64, rounded, stats_bounds,
                     strided)

pytestmark = pytest.mark.gpu


def _dobb():
    import block_eigenbasis_preconditioning_gb300 as d
    return d


def _logits(rows, vocab, seed, dtype, std=3.0):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, vocab)) * std
    return rounded(x, dtype), rng.integers(0, vocab, rows)


def _forward(x, t, dtype, scale=1.0, k=0, extra=0, offset=0, token_dtype=torch.int64, **kw):
    xd = strided(x, dtype, extra, offset)
    td = torch.from_numpy(np.asarray(t)).to("cuda", token_dtype)
    return xd, td, _dobb().log_probs(xd, td, scale=scale, top_k=k, **kw)


def _check_forward(x, t, r, scale, k):
    f = L.log_probs(x, t, scale, k)
    eS, eH = stats_bounds(x, scale, f)
    assert_close(np64(r.row_max), f["row_max"], 0.0, "row_max")
    assert_close(np64(r.log_sum), f["log_sum"], eS, "log_sum")
    assert_close(np64(r.lse), f["lse"], eS + 3 * U * np.abs(np.where(np.isfinite(f["lse"]), f["lse"], 0)) +
                 2 * U * np.abs(np.where(np.isfinite(f["row_max"]), f["row_max"] * scale, 0)), "lse")
    with np.errstate(invalid="ignore"):
        w = np.where(np.isfinite(f["logp"]), f["logp"] + f["log_sum"], 0.0)
        assert_close(np64(r.logp), f["logp"], np.where(np.asarray(t) < 0, 0.0, logp_bound(w, np.where(np.isfinite(f["log_sum"]), f["log_sum"], 0), eS)), "logp")
    if r.entropy is not None:
        assert_close(np64(r.entropy), f["entropy"], eH, "entropy")
    if k:
        assert np.array_equal(r.top_ids.cpu().numpy(), f["top_ids"]), "top_ids"
        with np.errstate(invalid="ignore"):
            ls = np.where(np.isfinite(f["log_sum"]), f["log_sum"], 0)[:, None]
            w = np.where(np.isfinite(f["top_logp"]), f["top_logp"] + ls, 0.0)
            assert_close(np64(r.top_logp), f["top_logp"], logp_bound(w, ls, eS[:, None]), "top_logp")
    return f, eS, eH


SIZES = [(1, 1), (1, 2), (3, 7), (2, 31), (5, 33), (4, 255), (2, 256), (3, 257), (2, 1000), (7, 4099), (1, 50257),
         (3, 50257), (170, 513), (40, 9001), (1, 128256), (20, 30000)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,vocab", SIZES)
def test_forward_sizes(rows, vocab, dtype):
    x, t = _logits(rows, vocab, rows * 7 + vocab, dtype)
    k = min(vocab, 5)
    _, _, r = _forward(x, t, dtype, 0.8, k)
    _check_forward(x, t, r, 0.8, k)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("extra,offset,token_dtype", [(0, 1, torch.int32), (1, 0, torch.int64), (47, 3, torch.int32),
                                                       (8, 8, torch.int64), (5, 7, torch.int64)])
def test_forward_strides_offsets_and_token_types(dtype, extra, offset, token_dtype):
    x, t = _logits(9, 2051, 11, dtype)
    _, _, r = _forward(x, t, dtype, 1.0, 3, extra, offset, token_dtype)
    _check_forward(x, t, r, 1.0, 3)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("k", [1, 2, 8, 31, 32])
@pytest.mark.parametrize("vocab", [32, 100, 5000, 70001])
def test_alternatives_with_many_ties(dtype, k, vocab):
    """Logits on few levels: almost every place of the answer is a tie."""
    rng = np.random.default_rng(vocab + k)
    x = rng.integers(-2, 3, (4, vocab)).astype(np.float32)
    x[1] = 0.0
    x[1, ::2] = -0.0                      # equal to 0
    x[2] = -np.inf
    x[2, vocab // 2] = 1.0                # one token is possible
    x[3] = np.sort(x[3])                  # the largest come last
    t = rng.integers(0, vocab, 4)
    _, _, r = _forward(x, t, dtype, 1.0, k)
    _check_forward(x, t, r, 1.0, k)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("vocab,k", [(1, 1), (5, 5), (33, 32), (700, 9), (2050, 32), (4093, 3)])
def test_many_short_rows(dtype, vocab, k):
    rng = np.random.default_rng(vocab)
    rows = 640
    x = rounded(rng.standard_normal((rows, vocab)) * 2, dtype)
    x[1::5] = rng.integers(-1, 2, x[1::5].shape)          # ties
    x[2::10] = -np.inf
    x[3::10, 1:] = float(torch.finfo(TORCH[dtype]).min)
    x[4::10, vocab // 2] = np.nan
    x[5::10, : vocab // 2] = -np.inf
    t = rng.integers(-1, vocab, rows)
    _, _, r = _forward(x, t, dtype, 0.9, k, 1, 1)
    _check_forward(x, t, r, float(np.float32(0.9)), k)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("k", [1, 9, 32])
def test_alternatives_with_many_ties_over_many_long_rows(dtype, k):
    rng = np.random.default_rng(k)
    rows, vocab = 310, 17003
    x = rng.integers(-2, 3, (rows, vocab)).astype(np.float32)
    x[1::4] = 0.0
    x[2::4] = -np.inf
    x[2::8, 5::1000] = 1.0                # 17 tokens are possible
    x[3::4] = rounded(rng.standard_normal((len(x[3::4]), vocab)), dtype)
    x[3::8, 77::256 * 8] += 8.0           # the largest sit far apart in one stride
    x[3::8] = rounded(x[3::8], dtype)
    x[7::16, :600] = 9.0 + np.arange(600) # and one next to the other
    x[7::16] = rounded(x[7::16], dtype)
    x[0] = np.sort(x[0])
    t = rng.integers(0, vocab, rows)
    _, _, r = _forward(x, t, dtype, 1.0, k, 3, 1)
    _check_forward(x, t, r, 1.0, k)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows", [1, 6, 400])
@pytest.mark.parametrize("vocab", [37, 4000, 40001])
def test_masked_rows_lowest_values_and_non_finite(dtype, rows, vocab):
    rng = np.random.default_rng(vocab)
    x = rounded(rng.standard_normal((rows, vocab)) * 2, dtype)
    low = float(torch.finfo(TORCH[dtype]).min)
    t = rng.integers(0, vocab, rows)
    kinds = [lambda r: r.fill(-np.inf), lambda r: r.fill(low), lambda r: r.__setitem__(slice(1, None), low),
             lambda r: r.__setitem__(slice(0, vocab - 1), -np.inf), lambda r: r.__setitem__(vocab // 3, np.nan),
             lambda r: r.__setitem__(vocab // 2, np.inf), lambda r: r.__setitem__(slice(0, None, 2), -np.inf)]
    for i in range(rows):
        kinds[(i + (rows == 1) * vocab) % len(kinds)](x[i])
    t[::5] = -100
    k = 4
    xd, td, r = _forward(x, t, dtype, 1.0, k)
    f, eS, eH = _check_forward(x, t, r, 1.0, k)
    g, h, l = (rng.standard_normal(rows).astype(np.float32) for _ in range(3))
    d = np64(_dobb().log_probs_backward(xd, td, r, torch.from_numpy(g).cuda(), grad_entropy=torch.from_numpy(h).cuda(),
                                        grad_lse=torch.from_numpy(l).cuda()))
    want = L.log_probs_backward(x, t, g, h, l)
    bad = np.isnan(f["log_sum"])
    assert np.isnan(d[bad]).all(axis=1).all()
    b = grad_bound(x, t, f, eS, eH, g, h, l, 1.0, dtype)
    assert_close(d[~bad], want[~bad], b[~bad] + HALF_UNIT[dtype] * np.abs(want[~bad]) * (1 + 1e-3) + TINY[dtype], "dlogits")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows", [1, 9, 330])
@pytest.mark.parametrize("vocab", [50, 20011])
@pytest.mark.parametrize("scale", [1.0, 1.25])
def test_finite_masks_and_huge_logits(dtype, rows, vocab, scale):
    """Masks that are ordinary numbers, alone in a row and next to others, and
    logits so large that their product with log2(e) rounds by more than one."""
    rng = np.random.default_rng(vocab)
    x = rng.standard_normal((rows, vocab)).astype(np.float32)
    masks = [-1e9, -1e10, -1e30, -1.4e9, -1.6e9, 2.5e9, 7e20, -3e38]
    for i in range(rows):
        v = np.float32(masks[i % len(masks)])
        kind = (i // len(masks) + i) % 3
        if kind == 0:
            x[i] = v                                     # nothing else
        elif kind == 1:
            x[i, : vocab - 1] = v                        # one entry is not masked
        else:
            x[i, rng.random(vocab) < 0.5] = v
        if abs(v) < 1e11:
            x[i, 3:9] *= np.float32(1 + 2.0 ** -20)      # neighbours, some units away
    x = rounded(x, dtype)
    t = rng.integers(0, vocab, rows)
    xd, td, r = _forward(x, t, dtype, scale, 4)
    f, eS, eH = _check_forward(x, t, r, float(np.float32(scale)), 4)
    g = rng.standard_normal(rows).astype(np.float32)
    d = np64(_dobb().log_probs_backward(xd, td, r, torch.from_numpy(g).cuda(), grad_entropy=torch.from_numpy(g).cuda()))
    want = L.log_probs_backward(x, t, g, g, None, float(np.float32(scale)))
    b = grad_bound(x, t, f, eS, eH, g, g, None, scale, dtype)
    assert_close(d, want, b + HALF_UNIT[dtype] * np.abs(want) * (1 + 1e-3) + TINY[dtype], "dlogits")


def test_tokens_outside_the_vocabulary_set_the_flag():
    x, _ = _logits(5, 300, 1, "f32")
    t = np.array([0, -1, 300, 7, 1 << 20])
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    xd, td, r = _forward(x, t, "f32", flags=flags)
    _check_forward(x, t, r, 1.0, 0)
    assert int(flags) == 16
    d = _dobb().log_probs_backward(xd, td, r, torch.ones(5, device="cuda"))
    assert not d[1].any() and not d[2].any() and not d[4].any() and d[0].any()
    flags.zero_()
    _forward(x, np.array([0, -1, -5, 7, 299]), "f32", flags=flags)
    assert int(flags) == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,vocab,extra,offset", [(1, 1, 0, 0), (3, 5, 0, 1), (1, 50257, 0, 0), (9, 4097, 3, 5), (64, 1024, 0, 0),
                                                     (300, 771, 0, 0), (2, 128256, 0, 0)])
@pytest.mark.parametrize("with_h,with_l,scale", [(False, False, 1.0), (True, False, 1.0), (True, True, 0.7)])
def test_gradient(dtype, rows, vocab, extra, offset, with_h, with_l, scale):
    rng = np.random.default_rng(rows + vocab)
    x, t = _logits(rows, vocab, rows + vocab, dtype)
    t[rows // 2] = -1 if rows > 2 else t[rows // 2]
    xd, td, r = _forward(x, t, dtype, scale, 0, extra, offset)
    f = L.log_probs(x, t, scale)
    eS, eH = stats_bounds(x, scale, f)
    g, h, l = (rng.standard_normal(rows).astype(np.float32) for _ in range(3))
    cu = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    kw = dict(grad_entropy=cu(h) if with_h else None, grad_lse=cu(l) if with_l else None)
    d = _dobb().log_probs_backward(xd, td, r, cu(g), **kw)
    want = L.log_probs_backward(x, t, g, h if with_h else None, l if with_l else None, scale)
    b = grad_bound(x, t, f, eS, eH, g, h if with_h else None, l if with_l else None, scale, dtype)
    b = b + HALF_UNIT[dtype] * np.abs(want) * (1 + 1e-3) + TINY[dtype]
    assert_close(np64(d), want, b, "dlogits")
    # into a strided matrix, and in place: the same bits; nothing between the rows is touched
    o = strided(np.zeros_like(x), dtype, 11, 3)
    _dobb().log_probs_backward(xd, td, r, cu(g), out=o, **kw)
    assert torch.equal(o, d)
    assert torch.isnan(o.as_strided((rows, 11), (o.stride(0), 1), o.storage_offset() + vocab)[: rows - 1]).all()
    _dobb().log_probs_backward(xd, td, r, cu(g), out=xd, **kw)
    assert torch.equal(xd, d)


def test_gradient_against_differences():
    """Central differences of the fp64 forward: with step 1e-4 they are off by
    about step^2 times the third derivative (< 10) = 1e-7; the kernel's own
    bound is below that here."""
    x, t = _logits(3, 40, 5, "f32", 2.0)
    g, h, l = np.random.default_rng(6).standard_normal((3, 3)).astype(np.float32)
    cu = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    xd, td, r = _forward(x, t, "f32", 0.9)
    d = np64(_dobb().log_probs_backward(xd, td, r, cu(g), grad_entropy=cu(h), grad_lse=cu(l)))

    def loss(y):
        f = L.log_probs(y, t, 0.9)
        return float((g * f["logp"] + h * f["entropy"] + l * f["lse"]).sum())

    for i in range(3):
        for j in range(40):
            a, b = x.astype(np.float64), x.astype(np.float64)
            a[i, j] += 1e-4
            b[i, j] -= 1e-4
            assert abs(d[i, j] - (loss(a) - loss(b)) / 2e-4) < 2e-5


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_past_32_bit_offsets(dtype):
    """Rows whose element offsets pass 2^31 (a long row stride over few rows)."""
    vocab, stride, rows = 1003, (1 << 30) + 3, 3
    buf = torch.empty(2 * stride + vocab, dtype=TORCH[dtype], device="cuda")
    xd = torch.as_strided(buf, (rows, vocab), (stride, 1))
    x, t = _logits(rows, vocab, 2, dtype)
    xd.copy_(torch.from_numpy(x).cuda())
    td = torch.from_numpy(t).cuda()
    r = _dobb().log_probs(xd, td, top_k=2)
    f, eS, eH = _check_forward(x, t, r, 1.0, 2)
    g = torch.ones(rows, device="cuda")
    _dobb().log_probs_backward(xd, td, r, g, out=xd)
    want = L.log_probs_backward(x, t, np.ones(rows))
    b = grad_bound(x, t, f, eS, eH, np.ones(rows), None, None, 1.0, dtype)
    assert_close(np64(xd), want, b + HALF_UNIT[dtype] * np.abs(want) * (1 + 1e-3) + TINY[dtype], "dlogits")


def test_no_rows_other_stream_and_repeatability():
    d = _dobb()
    e = d.log_probs(torch.empty(0, 77, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda"), top_k=3)
    assert e.logp.shape == (0,) and e.top_ids.shape == (0, 3)
    assert d.log_probs_backward(torch.empty(0, 77, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda"), e,
                                torch.empty(0, device="cuda")).shape == (0, 77)
    x, t = _logits(33, 50257, 3, "bf16")
    xd, td, r = _forward(x, t, "bf16", 1.0, 6)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    q = d.log_probs(xd, td, top_k=6, stream=side)
    side.synchronize()
    for a, b in zip(r[:-1], q[:-1]):
        assert torch.equal(a, b)
    assert d.log_probs(xd, td, entropy=False).entropy is None


def test_a_result_for_other_rows_is_refused():
    d = _dobb()
    xd, td, r = _forward(*_logits(3, 50, 1, "f32"), "f32", 1.0, 0)
    g = torch.ones(2, device="cuda")
    for bad in (r, r._replace(stats=r.stats[:1, :2].contiguous()), r._replace(stats=r.stats[:, :2]),
                r._replace(stats=r.stats[:2, :2].double().contiguous())):
        with pytest.raises(ValueError):
            d.log_probs_backward(xd[:2], td[:2], bad, g)
