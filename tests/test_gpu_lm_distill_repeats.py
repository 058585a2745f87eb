"""Distillation: a teacher's id that comes twice in a row, wherever its two places are, and ids whose hashes
meet.  The bounds are those of test_gpu_lm_distill."""
import numpy as np
import pytest

from test_gpu_lm_distill import _check, _inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("k", [2, 32, 33, 64, 65, 256])
def test_an_id_at_any_two_places(k):
    rows, vocab = 600, 1500
    x, ids, t, g = _inputs(rows, vocab, k, "f32", "f32", 40 + k)
    rng = np.random.default_rng(k)
    for r in range(rows):
        i, j = rng.permutation(k)[:2]
        if r % 3 == 0:  # neighbours, and the two ends of a round
            i, j = [(0, 1), (k - 2, k - 1), (0, min(k, 32) - 1), (min(31, k - 1), min(32, k - 1) if k > 32 else 0)][r // 3 % 4]
        ids[r, i] = ids[r, j]
    _check(x, ids, t, g, "f32", "f32")


def test_ids_whose_hashes_are_near():
    """Neighbouring and evenly spread ids, none of them twice, one of them twice, and all of one value."""
    k, vocab = 256, 140000
    x, ids, t, g = _inputs(12, vocab, k, "bf16", "f32", 41)
    for r, step in enumerate((1, 2, 3, 233, 377, 256, 512, 13, 17, 64)):
        ids[r] = 5 + step * np.arange(k)
        ids[r, 1::2] = ids[r, 1::2][::-1]
        if r % 2:
            ids[r, 200] = ids[r, 7]
    ids[10] = vocab - 1
    ids[11, 32:] = np.tile(ids[11, :32], 7)
    _check(x, ids, t, g, "bf16", "f32")
