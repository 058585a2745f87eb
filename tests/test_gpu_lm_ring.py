"""Log probabilities of many long rows, which are copied in ahead of the
arithmetic: thousands of rows, so that every block takes several in turn and
each of its buffers is used again and again, and the bounded waits for the copies.

The definition is evaluated in fp64 on the device, row by row the same as
oracle/lm.py's; the bounds are those of lm_util, vectorised."""
import time

import pytest
import torch

from lm_util import TORCH, U, chain

pytestmark = pytest.mark.gpu

INF = float("inf")


def _dobb():
    import block_eigenbasis_preconditioning_gb300 as d
    return d


def _logits(rows, vocab, dtype, extra, offset, seed):
    """Rows of every kind, in an order that no power of two repeats."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.rand(*s, device="cuda", generator=gen)  # noqa: E731
    x = torch.randn(rows, vocab, device="cuda", generator=gen) * 3
    x[1::7] = torch.randint(-2, 3, x[1::7].shape, device="cuda", generator=gen).float()   # ties
    x[2::11] = -INF
    x[3::13, vocab // 3] = float("nan")
    x[4::17, vocab // 2] = INF
    x[5::19].masked_fill_(rand(*x[5::19].shape) < 0.5, -INF)
    x[6::23] = float(torch.finfo(TORCH[dtype]).min)
    x[7::29, 1:] = -1e30
    x[8::31, 40:300] = 11.0 + torch.arange(260, device="cuda") / 16.0                     # the largest side by side
    x[9::37] = torch.sort(x[9::37], dim=1).values
    x[10::41, 3:] = -INF
    buf = torch.full((offset + rows * (vocab + extra),), float("nan"), device="cuda", dtype=TORCH[dtype])
    v = buf[offset:].view(rows, vocab + extra)[:, :vocab]
    v.copy_(x)
    t = torch.randint(0, vocab, (rows,), device="cuda", generator=gen)
    t[::9] = -1
    return v, t


def _definition(x, t, scale, k):
    """logp, lse, entropy, row_max, log_sum, ids, alternatives and the bounds
    of log_sum and the entropy, fp64."""
    x = x.double()
    v = x.shape[1]
    nan = x.isnan()
    m = torch.where(nan, -INF, x).amax(1)
    bad = nan.any(1) | (m == INF)
    empty = ~bad & (m == -INF)
    fine = ~bad & ~empty
    w = torch.where(fine[:, None], scale * (x - m[:, None]), 0.0)
    e = torch.where(fine[:, None], w.exp(), 0.0)
    log_sum = torch.where(fine, e.sum(1).log(), torch.where(empty, -INF, float("nan")))
    lp = torch.where(fine[:, None], w - log_sum[:, None], log_sum[:, None])
    p = torch.where(fine[:, None], lp.exp(), 0.0)
    ent = torch.where(fine, -torch.where(p > 0, p * lp, 0.0).sum(1), torch.where(empty, 0.0, float("nan")))
    lse = torch.where(fine, scale * m + log_sum, log_sum)
    logp = torch.where(t < 0, 0.0, lp.gather(1, t.clamp(min=0)[:, None])[:, 0])
    ids = (x + 0.0).sort(dim=1, descending=True, stable=True).indices[:, :k]
    pw = torch.where(p > 0, p * -w, 0.0)
    W, W2 = pw.sum(1), torch.where(p > 0, pw * -w, 0.0).sum(1)
    ls = torch.where(fine, log_sum, 0.0).abs()
    rel = U * (2 * W + 8 + chain(v))
    eS = rel + 3 * U * ls + U
    eH = eS + U * (2 * W2 + (10 + chain(v)) * W) + W * rel + 3 * U * (W + ls)
    return dict(logp=logp, lse=lse, entropy=ent, row_max=m, log_sum=log_sum, ids=ids, alt=lp.gather(1, ids), eS=eS, eH=eH, ls=ls)


def _close(got, want, bound, what):
    got = got.double()
    want = torch.where(want.abs() > torch.finfo(torch.float32).max, want.sign() * INF, want)
    fine = want.isfinite()
    assert torch.equal(got.isnan(), want.isnan()), what
    rest = ~fine & ~want.isnan()
    assert torch.equal(got[rest], want[rest]), what
    err = (got - want).abs()[fine]
    assert bool((err <= bound.expand_as(want)[fine]).all()), f"{what}: {float(err.max())}"


CASES = [("f32", 3001, 4100, 1, 1), ("f32", 2111, 9001, 0, 0), ("bf16", 3001, 17003, 3, 5), ("bf16", 4001, 5003, 0, 0)]


@pytest.mark.parametrize("dtype,rows,vocab,extra,offset", CASES)
@pytest.mark.parametrize("k", [0, 5, 32])
@pytest.mark.parametrize("entropy", [True, False])
def test_rows_in_turn(dtype, rows, vocab, extra, offset, k, entropy):
    scale = 0.75
    x, t = _logits(rows, vocab, dtype, extra, offset, vocab + k)
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = _dobb().log_probs(x, t, scale=scale, top_k=k, entropy=entropy, flags=flags)
    f = _definition(x, t, scale, k)
    fin = lambda a: torch.where(a.isfinite(), a, 0.0).abs()  # noqa: E731
    _close(r.row_max, f["row_max"], torch.zeros_like(f["eS"]), "row_max")
    _close(r.log_sum, f["log_sum"], f["eS"], "log_sum")
    _close(r.lse, f["lse"], f["eS"] + 3 * U * fin(f["lse"]) + 2 * U * scale * fin(f["row_max"]), "lse")
    some = f["eS"] + U * (4 * fin(f["logp"]) + 6 * f["ls"]) + U
    _close(r.logp, f["logp"], torch.where(t < 0, 0.0, some), "logp")
    if entropy:
        _close(r.entropy, f["entropy"], f["eH"], "entropy")
    if k:
        assert torch.equal(r.top_ids.long(), f["ids"])
        _close(r.top_logp, f["alt"], f["eS"][:, None] + U * (4 * fin(f["alt"]) + 6 * f["ls"][:, None]) + U, "top_logp")
    assert int(flags) == 0
    same = lambda a, b: a is b is None or torch.equal(a.nan_to_num(7e7), b.nan_to_num(7e7))  # noqa: E731
    for _ in range(3):
        q = _dobb().log_probs(x, t, scale=scale, top_k=k, entropy=entropy)
        assert all(same(a, b) for a, b in zip(r[:-1], q[:-1]))


@pytest.mark.parametrize("dtype,vocab", [("f32", 9001), ("bf16", 17003)])
@pytest.mark.parametrize("loaded", [0, 1000, 2999, 3001])
@pytest.mark.parametrize("entropy,k,with_flags", [(True, 5, True), (False, 0, False), (True, 32, False)])
def test_rows_that_a_wait_gave_up_on_hold_nan(dtype, vocab, loaded, entropy, k, with_flags):
    """Rows that are never copied in: the waits run out, those rows hold NaN (but
    logp where there is no token) and so does their gradient, whether or not there
    are flags, and the next call is right again."""
    from block_eigenbasis_preconditioning_gb300 import binding
    d, lib, rows = _dobb(), binding.load_library(), 3001
    gen = torch.Generator(device="cuda").manual_seed(loaded + k)
    x = torch.randn(rows, vocab, device="cuda", generator=gen).to(TORCH[dtype])
    t = torch.randint(-1, vocab, (rows,), device="cuda", generator=gen)
    want = d.log_probs(x, t, top_k=k, entropy=entropy)
    f = torch.full((5, rows), 7.0, device="cuda")
    ids = torch.full((rows, k), 7, device="cuda", dtype=torch.int32)
    alt = torch.full((rows, k), 7.0, device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    p = [f[i].data_ptr() for i in range(5)]
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    st = lib.dobb_selftest_log_probs_timeout(
        x.data_ptr(), binding.DTYPES[dtype], rows, vocab, vocab, t.data_ptr(), 8, 1.0, k, p[2], p[3], p[0], p[1],
        p[4] if entropy else None, ids.data_ptr() if k else None, alt.data_ptr() if k else None,
        flags.data_ptr() if with_flags else None, torch.cuda.current_stream().cuda_stream, loaded, 50_000_000)
    assert st == 0
    torch.cuda.synchronize()
    assert time.perf_counter() - t0 < 5.0
    got = d.LogProbs(f[2], f[3], f[4] if entropy else None, ids if k else None, alt if k else None, f, 1.0)
    for a, b in zip(got[:5], want[:5]):
        if a is not None:
            assert torch.equal(a[:loaded], b[:loaded])
            lost = a[loaded:]
            assert bool((lost == -1).all() if a is ids else (lost.isnan() | (lost == 0.0) & (t[loaded:] < 0)).all() if a is got.logp
                        else lost.isnan().all())
    assert torch.equal(got.row_max[:loaded], want.row_max[:loaded]) and bool(f[:2, loaded:].isnan().all())
    assert entropy or bool((f[4] == 7.0).all())
    assert int(flags) == (binding.FLAG_TIMEOUT if with_flags and loaded < rows else 0)
    g = torch.ones(rows, device="cuda")
    dx = d.log_probs_backward(x, t, got, g)
    assert bool(dx[loaded:].isnan().all()) and torch.equal(dx[:loaded], d.log_probs_backward(x, t, want, g)[:loaded])
    again = d.log_probs(x, t, top_k=k, entropy=entropy)
    for a, b in zip(again[:5], want[:5]):
        assert (a is None and b is None) or torch.equal(a, b)


def test_limits_of_the_self_test():
    from block_eigenbasis_preconditioning_gb300 import binding
    lib = binding.load_library()
    x, t = torch.zeros(700, 9000, device="cuda"), torch.zeros(700, dtype=torch.int64, device="cuda")
    f = torch.full((4, 700), 7.0, device="cuda")
    p = [f[i].data_ptr() for i in range(4)]

    def call(rows, loaded, limit):
        return lib.dobb_selftest_log_probs_timeout(x.data_ptr(), 0, rows, 9000, 9000, t.data_ptr(), 8, 1.0, 0, *p, None, None, None,
                                                   None, torch.cuda.current_stream().cuda_stream, loaded, limit)

    assert call(700, 701, 10 ** 6) == call(700, -1, 10 ** 6) == call(700, 0, 0) == call(700, 0, 6 * 10 ** 9) == 1
    assert call(10, 5, 10 ** 6) == 6 and b"no copies" in lib.dobb_last_error()
    torch.cuda.synchronize()
    assert bool((f == 7.0).all())
