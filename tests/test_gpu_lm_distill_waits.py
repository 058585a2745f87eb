"""Rows of distillation that a wait gave up on: copies that one block of a cluster never makes, bounded waits that
run out, NaN and the flag; the rows before are whole, and so is the next call."""
import time

import numpy as np
import pytest
import torch

from lm_util import dev
from test_gpu_lm_distill import _inputs

pytestmark = pytest.mark.gpu


def _call(x, ids, t, g, loaded, late_part, limit_ns, with_flags=True):
    from block_eigenbasis_preconditioning_gb300 import binding
    rows, vocab = x.shape
    f = torch.full((3, rows), 7.0, device="cuda")
    out, flags = torch.full_like(x, 7.0), torch.zeros(1, dtype=torch.int32, device="cuda")
    p = [f[i].data_ptr() for i in range(3)]
    st = binding.load_library().dobb_selftest_distill_timeout(
        x.data_ptr(), {torch.float32: 0, torch.bfloat16: 1}[x.dtype], rows, vocab, vocab, ids.data_ptr(), 4, t.data_ptr(), 0, t.shape[1], 1.0, 1.0,
        p[2], p[0], p[1], g.data_ptr(), out.data_ptr(), vocab, flags.data_ptr() if with_flags else None,
        torch.cuda.current_stream().cuda_stream, loaded, late_part, limit_ns)
    return st, f, out, flags


def _data(rows, vocab, xt, seed):
    x, ids, t, g = _inputs(rows, vocab, 9, xt, "f32", seed)
    return dev(x, xt), torch.from_numpy(ids.astype(np.int32)).cuda(), dev(t, "f32"), dev(g, "f32")


@pytest.mark.parametrize("xt,rows,vocab,part", [("f32", 120, 150000, 0), ("f32", 120, 150000, 1), ("f32", 120, 150000, 5), ("bf16", 400, 98304, 1),
                                                ("bf16", 700, 20000, 0)])
@pytest.mark.parametrize("loaded", [0, 60, -1])
def test_the_flag_and_nan_whichever_block_is_late(xt, rows, vocab, part, loaded):
    import block_eigenbasis_preconditioning_gb300 as d
    from block_eigenbasis_preconditioning_gb300 import binding
    loaded = rows if loaded < 0 else loaded
    args = _data(rows, vocab, xt, 50 + part)
    args[1][3] = args[1][-2] = -1  # rows without entries
    want = d.distill(*args[:3], grad_loss=args[3])
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    st, f, out, flags = _call(*args, loaded, part, 50_000_000, with_flags=part != 5 or loaded != 0)
    assert st == 0
    torch.cuda.synchronize()
    assert time.perf_counter() - t0 < 5.0
    assert torch.equal(f[:, :loaded], want.stats[:, :loaded]) and torch.equal(out[:loaded], want.grad[:loaded])
    assert bool(f[:2, loaded:].isnan().all())
    assert bool(f[2, loaded:].isnan().all()) and bool(out[loaded:].isnan().all())
    assert int(flags) == (binding.FLAG_TIMEOUT if loaded < rows and (part != 5 or loaded != 0) else 0)
    again = d.distill(*args[:3], grad_loss=args[3])
    assert torch.equal(again.stats, want.stats) and torch.equal(again.grad, want.grad)


def test_limits_of_the_self_test():
    from block_eigenbasis_preconditioning_gb300 import binding
    args = _data(10, 60000, "f32", 60)  # (stretches of 8192 entries at least: seven blocks)
    for loaded, part, limit in ((11, 0, 10 ** 6), (-1, 0, 10 ** 6), (5, 0, 0), (5, 0, 6 * 10 ** 9), (5, 7, 10 ** 6), (5, -1, 10 ** 6)):
        st, f, out, flags = _call(*args, loaded, part, limit)
        assert st == 1
        torch.cuda.synchronize()
        assert bool((f == 7.0).all()) and bool((out == 7.0).all()) and int(flags) == 0
    st, f, out, _ = _call(*_data(2, 300001, "f32", 61), 1, 0, 10 ** 6)
    assert st == 6 and b"no copies" in binding.load_library().dobb_last_error()
