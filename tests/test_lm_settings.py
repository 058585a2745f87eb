"""Settings of distillation, sampling and layer norm: numbers of any kind are taken, what is none is refused
with ValueError, before any device is asked for."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import block_eigenbasis_preconditioning_gb300 as dobb

NOT_NUMBERS = ("0.5", "a", None, [1.0], 1j, object())


def _calls(device):
    g = torch.Generator().manual_seed(3)
    x, e = torch.randn(5, 40, generator=g).to(device), torch.rand(5, 40, generator=g).to(device) + 0.1
    ids, t = torch.arange(15).view(5, 3).to(device), torch.randn(5, 3, generator=g).to(device)
    return {"scale": lambda v: dobb.sample(x, e, scale=v), "top_p": lambda v: dobb.sample(x, e, top_p=v), "min_p": lambda v: dobb.sample(x, e, min_p=v),
            "top_k": lambda v: dobb.sample(x, e, top_k=v), "eps": lambda v: dobb.layer_norm(x, eps=v),
            "distill's scale": lambda v: dobb.distill(x, ids, t, scale=v, teacher_scale=1.0), "teacher_scale": lambda v: dobb.distill(x, ids, t, teacher_scale=v)}


@pytest.mark.parametrize("name", list(_calls("cpu")))
def test_what_is_no_number(name):
    call = _calls("cpu")[name]
    for v in NOT_NUMBERS + ((50.0, np.float32(3), Fraction(3)) if name == "top_k" else ()):
        if v is None and name == "teacher_scale":
            continue  # (the scale's)
        with pytest.raises(ValueError, match="number"):
            call(v)


@pytest.mark.gpu
def test_numbers_of_other_kinds():
    calls = _calls("cuda")
    for name, call in calls.items():
        plain, others = (2, (np.int64(2), np.int32(2), np.uint8(2))) if name == "top_k" else (0.5, (np.float32(0.5), np.float64(0.5), Fraction(1, 2), np.float16(0.5)))
        want = call(plain)
        for v in others:
            assert all(torch.equal(a, b) for a, b in zip(call(v), want) if isinstance(a, torch.Tensor)), (name, type(v))
