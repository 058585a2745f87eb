"""Log probabilities of many long rows, which are copied in ahead of the
arithmetic: the bounded waits for the copies."""
import time

import pytest
import torch

from lm_util import TORCH

pytestmark = pytest.mark.gpu


def _dobb():
    import block_eigenbasis_preconditioning_gb300 as d
    return d


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
