"""The native call with tensors that have no memory: an error of the call, as the interpreter's way gives it, and the
interpreter's lock is held again."""
import subprocess
import sys

import pytest

PROGRAM = """
import threading, torch
import block_eigenbasis_preconditioning_gb300 as dobb
from torch._subclasses.fake_tensor import FakeTensorMode
real = [torch.randn(4, 64, device="cuda"), torch.ones(4, 64, device="cuda")]
stop, turns = threading.Event(), [0]
def other():
    while not stop.is_set():
        turns[0] += len([object() for _ in range(100)])
t = threading.Thread(target=other)
t.start()
mode = FakeTensorMode(allow_non_fake_inputs=True)
with mode:
    x, e, v = torch.empty(4, 64, device="cuda"), torch.empty(4, 64, device="cuda"), torch.empty(4, device="cuda")
    ids = torch.empty(4, 3, dtype=torch.int32, device="cuda")
    r = dobb.lm.LayerNorm(x, v, v)
calls = (lambda: dobb.layer_norm(x), lambda: dobb.layer_norm_backward(x, x, r), lambda: dobb.sample(x, e),
         lambda: dobb.distill(x, ids, e[:, :3].contiguous()), lambda: dobb.sample(real[0], e))
errors = 0
for inside in (False, True):
    for call in calls:
        for _ in range(20):
            try:
                if inside:
                    with mode:
                        call()
                else:
                    call()
            except Exception as err:
                assert not isinstance(err, AssertionError), err
                errors += 1
stop.set()
t.join()
torch.cuda.synchronize()
assert errors == 200, errors
assert torch.isfinite(dobb.layer_norm(real[0]).out).all() and turns[0] > 0
print("every call said no")
"""


@pytest.mark.gpu
def test_tensors_without_memory():
    # (a process of its own: an error raised without the lock ends it)
    r = subprocess.run([sys.executable, "-c", "import block_eigenbasis_preconditioning_gb300.lm\n" + PROGRAM], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "every call said no" in r.stdout, r.stdout + r.stderr
