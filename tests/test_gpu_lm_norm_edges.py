"""Layer norm of tensors that begin and end within 16 bytes, with more turns of every slot than there are
slots: what the producer writes by value is copied over later."""
import pytest

from test_gpu_lm_norm import _check, _inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("extra,offset", [(0, 1), (0, 3), (1, 2), (8, 5), (4, 4)])
@pytest.mark.parametrize("rows,dim", [(9000, 130), (3000, 1603), (2500, 1600), (700, 6002), (20000, 21)])
def test_many_turns_from_any_place(rows, dim, extra, offset):
    for xt in ("f32", "bf16"):
        _check(*_inputs(rows, dim, xt, "bf16", "f32", rows + offset), xt, "bf16", "f32", extra=extra, offset=offset)
