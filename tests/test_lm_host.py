"""Refusals of the language-model operators, without a GPU: the C entries
check everything before any device work (fake addresses), the Python calls
raise ValueError."""
import ctypes
import os
import re

import pytest
import torch

import block_eigenbasis_preconditioning_gb300 as dobb
from block_eigenbasis_preconditioning_gb300 import binding, lm

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 20        # a made-up device address


@pytest.fixture(scope="module")
def lib():
    return binding.load_library()


def _refused(lib, st, word, status=1):
    assert st == status and word.encode() in lib.dobb_last_error(), lib.dobb_last_error()


def _args(base, **change):
    a = dict(base)
    assert not set(change) - set(a)
    a.update(change)
    return list(a.values())


LP = dict(logits=P, dtype=0, rows=4, vocab=100, stride=100, tokens=P, token_bytes=8, scale=1.0, k=0, logp=P, lse=P, row_max=P,
          log_sum=P, entropy=P, ids=P, alt=P, flags=None, stream=None)
LPB = dict(logits=P, dtype=0, rows=4, vocab=100, stride=100, tokens=P, token_bytes=8, scale=1.0, row_max=P, log_sum=P, entropy=P,
           g=P, h=P, l=P, out=2 * P, ostride=100, stream=None)
EM = dict(weight=P, wdtype=0, vocab=100, dim=8, wstride=8, tokens=P, token_bytes=8, count=4, scale=1.0, out=P, odtype=0, ostride=8,
          flags=None, stream=None)
EB = dict(grad=P, gdtype=0, count=4, dim=8, gstride=8, tokens=P, token_bytes=8, vocab=100, scale=1.0, out=P, odtype=0, ostride=8,
          accumulate=0, flags=None, ws=P, ws_bytes=1 << 30, stream=None)
NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("change,word", [
    (dict(dtype=2), "dtype"), (dict(rows=-1), "rows"), (dict(vocab=0), "vocab"), (dict(vocab=1 << 31, stride=1 << 31), "vocab"),
    (dict(stride=99), "row_stride"), (dict(token_bytes=2), "token_bytes"), (dict(scale=0.0), "scale"), (dict(scale=-1.0), "scale"),
    (dict(scale=NAN), "scale"), (dict(scale=INF), "scale"), (dict(logits=None), "non-NULL"), (dict(tokens=None), "non-NULL"),
    (dict(logits=P + 2), "aligned"), (dict(tokens=P + 4), "aligned")])
def test_log_probs_refusals(lib, change, word):
    _refused(lib, lib.dobb_log_probs(*_args(LP, **change)), word)
    _refused(lib, lib.dobb_log_probs_backward(*_args(LPB, **change)), word)


def test_more_log_probs_refusals(lib):
    for change, word in ((dict(k=-1), "top_k"), (dict(k=33), "top_k"), (dict(k=6, vocab=5), "top_k"), (dict(logp=None), "logp"),
                         (dict(row_max=None), "row_max"), (dict(k=2, ids=None), "top_ids"), (dict(k=2, alt=None), "top_logp")):
        _refused(lib, lib.dobb_log_probs(*_args(LP, **change)), word)
    for change, word in ((dict(ostride=99), "out_stride"), (dict(g=None), "grad_logp"), (dict(out=None), "dlogits"),
                         (dict(entropy=None), "entropy"), (dict(out=P, ostride=101), "in place"), (dict(out=P + 1), "aligned")):
        _refused(lib, lib.dobb_log_probs_backward(*_args(LPB, **change)), word)
    # no rows: nothing to do, whatever the pointers
    assert lib.dobb_log_probs(*_args(LP, rows=0, logits=None, tokens=None, logp=None)) == 0
    assert lib.dobb_log_probs_backward(*_args(LPB, rows=0, out=None)) == 0


@pytest.mark.parametrize("change,word", [
    (dict(wdtype=3), "dtype"), (dict(odtype=-1), "dtype"), (dict(vocab=0), "vocab"), (dict(dim=0), "dim"), (dict(count=-1), "count"),
    (dict(wstride=7), "stride"), (dict(ostride=7), "stride"), (dict(token_bytes=1), "token_bytes"), (dict(scale=NAN), "scale"),
    (dict(scale=INF), "scale"), (dict(weight=None), "non-NULL"), (dict(out=None), "non-NULL"), (dict(tokens=None), "non-NULL"),
    (dict(out=P + 2), "aligned"), (dict(tokens=P + 2), "aligned")])
def test_embedding_refusals(lib, change, word):
    _refused(lib, lib.dobb_embedding(*_args(EM, **change)), word)


@pytest.mark.parametrize("change,word", [
    (dict(gdtype=3), "dtype"), (dict(odtype=-1), "dtype"), (dict(vocab=0), "vocab"), (dict(vocab=(1 << 30) + 1), "vocab"),
    (dict(dim=0), "dim"), (dict(count=-1), "count"), (dict(count=1 << 31), "count"), (dict(gstride=7), "stride"),
    (dict(ostride=7), "stride"), (dict(token_bytes=1), "token_bytes"), (dict(scale=NAN), "scale"), (dict(accumulate=2), "accumulate"),
    (dict(grad=None), "non-NULL"), (dict(out=None), "non-NULL"), (dict(tokens=None), "non-NULL"), (dict(out=P + 2), "aligned"),
    (dict(ws=None), "workspace"), (dict(ws=P + 16), "workspace")])
def test_embedding_gradient_refusals(lib, change, word):
    _refused(lib, lib.dobb_embedding_backward(*_args(EB, **change)), word)


def test_embedding_workspace(lib):
    need = lib.dobb_embedding_backward_bytes(4, 100, 8)
    assert need > 0
    _refused(lib, lib.dobb_embedding_backward(*_args(EB, ws_bytes=need - 1)), "smaller", 5)
    assert lib.dobb_embedding_backward_bytes(0, 100, 8) > 0
    assert lib.dobb_embedding_backward_bytes(-1, 100, 8) == 0 and b"count" in lib.dobb_last_error()
    assert lib.dobb_embedding_backward_bytes(4, 0, 8) == 0 and lib.dobb_embedding_backward_bytes(4, 10, 0) == 0


def _clip(lib, num=2, g=(P, P + 4096), gd=(0, 0), ne=(16, 16), max_norm=1.0, out=(P, P + 4096), od=(0, 0), stats=P, ws=P,
          ws_bytes=1 << 20):
    ptr = lambda v: None if v is None else (ctypes.c_void_p * len(v))(*v)  # noqa: E731
    i32 = lambda v: None if v is None else (ctypes.c_int32 * len(v))(*v)  # noqa: E731
    return lib.dobb_clip_grads(num, ptr(g), i32(gd), None if ne is None else (ctypes.c_int64 * len(ne))(*ne), max_norm, ptr(out),
                               i32(od), stats, None, ws, ws_bytes, None)


@pytest.mark.parametrize("change,word", [
    (dict(num=0), "num_tensors"), (dict(ne=None), "numel"), (dict(ne=(3, -1)), "numel[1]"), (dict(g=None), "non-NULL"),
    (dict(gd=None), "non-NULL"), (dict(od=None), "non-NULL"), (dict(max_norm=-1.0), "max_norm"), (dict(max_norm=NAN), "max_norm"),
    (dict(stats=None), "stats"), (dict(gd=(0, 2)), "tensor 1"), (dict(od=(5, 0)), "tensor 0"), (dict(g=(None, P)), "G[0]"),
    (dict(out=(P, None)), "G[1]"), (dict(g=(P, P + 2)), "aligned"), (dict(od=(1, 0)), "in place"), (dict(ws=None), "workspace"),
    (dict(ws=P + 8), "workspace")])
def test_clip_refusals(lib, change, word):
    _refused(lib, _clip(lib, **change), word)


def test_clip_workspace(lib):
    ne = (ctypes.c_int64 * 2)(16, 1 << 20)
    need = lib.dobb_clip_grads_bytes(2, ne)
    assert need > 0
    _refused(lib, _clip(lib, ne=(16, 1 << 20), ws_bytes=need - 1), "smaller", 5)
    assert lib.dobb_clip_grads_bytes(0, ne) == 0 and lib.dobb_clip_grads_bytes(2, None) == 0
    huge = (ctypes.c_int64 * 1)(1 << 62)
    assert lib.dobb_clip_grads_bytes(1, huge) == 0 and b"too many" in lib.dobb_last_error()


def test_names_match_the_header():
    hdr = open(os.path.join(ROOT, "include", "dobb.h")).read()
    d = dict(re.findall(r"#define (DOBB_[A-Z_]+) (\d+)", hdr))
    assert int(d["DOBB_FLAG_BAD_TOKEN"]) == binding.FLAG_BAD_TOKEN and int(d["DOBB_MAX_TOP_K"]) == lm.MAX_TOP_K
    assert dobb.log_probs is lm.log_probs and dobb.clip_grads is lm.clip_grads and dobb.embedding is lm.embedding


def test_python_refusals():
    x, t = torch.zeros(4, 9), torch.zeros(4, dtype=torch.int64)
    for call in (lambda: dobb.log_probs(x, t),                                   # not on a GPU
                 lambda: dobb.log_probs(x.half(), t), lambda: dobb.log_probs(x, t.float()), lambda: dobb.log_probs(x, t[:3]),
                 lambda: dobb.log_probs(x[0], t), lambda: dobb.log_probs(x.t(), t), lambda: dobb.log_probs(x, t, top_k=10),
                 lambda: dobb.log_probs(x, t, top_k=-1), lambda: dobb.log_probs(x[:1].expand(4, 9), t),
                 lambda: dobb.embedding(x, t), lambda: dobb.embedding(x.double(), t), lambda: dobb.embedding(x, t.short()),
                 lambda: dobb.embedding(x, t[::2]), lambda: dobb.embedding(x, t, out=x, out_dtype=torch.bfloat16),
                 lambda: dobb.embedding_backward(x, t), lambda: dobb.embedding_backward(x, t, accumulate=True, vocab=3),
                 lambda: dobb.embedding_backward(x, t[:3], 5), lambda: dobb.embedding_backward(x, t, 5),
                 lambda: dobb.clip_grads([], 1.0), lambda: dobb.clip_grads([x], -1.0), lambda: dobb.clip_grads([x], float("nan")),
                 lambda: dobb.clip_grads([x], 1.0, out=[]), lambda: dobb.grad_norm([x]), lambda: dobb.grad_norm([])):
        with pytest.raises(ValueError):
            call()


@pytest.mark.gpu
def test_python_refusals_on_the_gpu():
    x, t = torch.zeros(4, 9, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    r = dobb.log_probs(x, t, entropy=False)
    g = torch.zeros(4, device="cuda")
    for call in (lambda: dobb.log_probs(x, t.cpu()), lambda: dobb.log_probs_backward(x, t, r, g, grad_entropy=g),
                 lambda: dobb.log_probs_backward(x, t, r, g.double()), lambda: dobb.log_probs_backward(x, t, r, g[:3]),
                 lambda: dobb.log_probs_backward(x, t, r, g, out=x.bfloat16()), lambda: dobb.log_probs_backward(x, t, r, g, out=x[:3]),
                 lambda: dobb.embedding(x, t, out=torch.empty(4, 8, device="cuda")),
                 lambda: dobb.embedding(x, t, out=torch.empty(9, 4, device="cuda").t()),
                 lambda: dobb.embedding_backward(x, t, 7, out=torch.empty(6, 9, device="cuda")),
                 lambda: dobb.embedding_backward(x, t, 7, dtype=torch.float16),
                 lambda: dobb.clip_grads([x[:, ::2]], 1.0), lambda: dobb.clip_grads([x.half()], 1.0),
                 lambda: dobb.clip_grads([x], 1.0, out=[x.t()]), lambda: dobb.clip_grads([x], 1.0, out=[x.half()]),
                 lambda: dobb.clip_grads([x, x.cpu()], 1.0)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(binding.DobbError):
        dobb.embedding_backward(x, t, 0)
