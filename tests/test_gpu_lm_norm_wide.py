"""Layer norm at the widths where fewer rows of a block fit its shared memory."""
import pytest

from test_gpu_lm_norm import _check, _inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,dim", [(200, 14333), (200, 14336), (310, 14336), (153, 14337), (200, 8193), (200, 10240), (460, 12288), (200, 16384)])
def test_wide_rows_of_several_groups(rows, dim):
    for xt, gt, pt in (("f32", "bf16", "f32"), ("f32", "f32", "bf16"), ("bf16", "bf16", "bf16")):
        _check(*_inputs(rows, dim, xt, gt, pt, dim % 100), xt, gt, pt)
