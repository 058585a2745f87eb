"""The two ends of a language model, and its gradients before a step.

Log probabilities of given tokens (with entropy, the most likely alternatives
and the gradient with respect to the logits), the embedding lookup and its
gradient by sorted tokens, and the global gradient norm with clipping.  They
make and prepare the gradients that `Dobb.step` takes for the embedding and
the head.

Argument checks and memory only: all arithmetic runs in the CUDA kernels
behind include/dobb.h, which states the formulas, the empty rows, the padding
and the non-finite cases.  Results are new tensors unless `out` is given.
Every call is asynchronous on `stream` (default: the current stream of the
tensors' device); results and workspaces are allocated on that stream, and
tensors that were made on another one are kept alive until it has passed.
Arguments of the wrong kind, shape or place raise ValueError, values and
overlaps that the library refuses (a scale of 0, an empty vocabulary, a gradient
listed twice) raise DobbError, both before anything is launched.

Autograd does not see these calls: results are not part of its graph, and what
is written in place or into `out` does not raise a tensor's version.  The
gradients are calls of their own.
"""
from __future__ import annotations

import ctypes
from array import array
from operator import attrgetter
from typing import NamedTuple, Optional, Sequence

import torch

from .binding import check, load_library

_DTYPES = {torch.float32: 0, torch.bfloat16: 1}
_TOKEN_BYTES = {torch.int32: 4, torch.int64: 8}
MAX_TOP_K = 32


class LogProbs(NamedTuple):
    """Result of `log_probs`, one entry per row (the alternatives: one row of
    top_k).  stats, whose first two rows are row_max and log_sum, and scale are
    what `log_probs_backward` needs: lse = scale * row_max + log_sum."""
    logp: torch.Tensor
    lse: torch.Tensor
    entropy: Optional[torch.Tensor]
    top_ids: Optional[torch.Tensor]
    top_logp: Optional[torch.Tensor]
    stats: torch.Tensor
    scale: float

    @property
    def row_max(self) -> torch.Tensor:
        return self.stats[0]

    @property
    def log_sum(self) -> torch.Tensor:
        return self.stats[1]


class GradNorm(NamedTuple):
    """Result of `grad_norm` and `clip_grads`: the global norm, the factor the
    gradients were multiplied with, and every tensor's own norm, fp32 on the
    device."""
    norm: torch.Tensor
    scale: torch.Tensor
    norms: torch.Tensor


# A serving call on a few rows takes the GPU microseconds, so the checks below
# are plain comparisons and the raw stream is read without a Stream object
# (0.1 us against 2 us); messages are built only when a check fails.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _device(first: torch.Tensor, *others: Optional[torch.Tensor]) -> int:
    """Index of the CUDA device that all of the tensors are on."""
    index = first.get_device()
    if index < 0:
        raise ValueError(f"tensors must be on a CUDA device, got {first.device}")
    for t in others:
        if t is not None and t.get_device() != index:
            raise ValueError(f"all tensors must be on {first.device}, got one on {t.device}")
    return index


class _On:
    """Device and stream of a call that is not on the current ones: what is
    allocated inside comes from that stream, and the tensors it uses outlive
    the work on it."""

    def __init__(self, index: int, stream: Optional[torch.cuda.Stream], used):
        if stream is None:
            self.ctx = torch.cuda.device(index)
        else:
            if stream.device.index != index:
                raise ValueError(f"the stream is on {stream.device}, the tensors on cuda:{index}")
            self.ctx = torch.cuda.stream(stream)
            for t in used:
                if t is not None:
                    t.record_stream(stream)

    def __enter__(self):
        self.ctx.__enter__()

    def __exit__(self, *exc):
        self.ctx.__exit__(*exc)


def _elsewhere(index: int, stream: Optional[torch.cuda.Stream]) -> bool:
    return stream is not None or index != _current_device()


def _rows(t: torch.Tensor, name: str) -> int:
    """Row stride of a matrix whose rows are contiguous."""
    if t.dim() != 2:
        raise ValueError(f"{name} must be a matrix, got {t.dim()} dimensions")
    rows, cols = t.shape
    down, across = t.stride()
    if across != 1 and cols > 1:
        raise ValueError(f"{name} must have contiguous rows")
    if down < cols:
        if rows > 1:
            raise ValueError(f"{name} must not overlap itself")
        return cols
    return down


def _token_bytes(t: torch.Tensor) -> int:
    size = _TOKEN_BYTES.get(t.dtype)
    if size is None:
        raise ValueError(f"tokens must be int32 or int64, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError("tokens must be contiguous")
    return size


def _vector(t: Optional[torch.Tensor], n: int, name: str) -> Optional[int]:
    if t is None:
        return None
    if t.dtype != torch.float32 or not t.is_contiguous() or t.numel() != n:
        raise ValueError(f"{name} must be {n} contiguous float32 values")
    return t.data_ptr()


def _flags(flags: Optional[torch.Tensor]) -> Optional[int]:
    if flags is None:
        return None
    if flags.dtype not in (torch.int32, torch.uint32) or flags.numel() != 1:
        raise ValueError("flags must be one int32 or uint32")
    return flags.data_ptr()


def _float_dtype(dtype: torch.dtype, name: str) -> int:
    code = _DTYPES.get(dtype)
    if code is None:
        raise ValueError(f"{name} must be float32 or bfloat16, got {dtype}")
    return code


# ------------------------------------------------------------ log probabilities

def log_probs(logits: torch.Tensor, tokens: torch.Tensor, *, scale: float = 1.0, top_k: int = 0,
              entropy: bool = True, flags: Optional[torch.Tensor] = None,
              stream: Optional[torch.cuda.Stream] = None) -> LogProbs:
    """Log probability of tokens[r] under softmax(scale * logits[r]), with the
    row's entropy and its top_k most likely tokens.

    logits: (rows, vocab) float32 or bfloat16 with contiguous rows at any row
    stride; tokens: rows indices, int32 or int64, below 0 for none.  -inf
    logits are banned tokens."""
    stride = _rows(logits, "logits")
    dtype = _float_dtype(logits.dtype, "logits")
    rows, vocab = logits.shape
    token_bytes = _token_bytes(tokens)
    if tokens.numel() != rows:
        raise ValueError(f"{tokens.numel()} tokens for {rows} rows")
    if not 0 <= top_k <= min(MAX_TOP_K, vocab):
        raise ValueError(f"top_k must lie in [0, min({MAX_TOP_K}, vocab)], got {top_k}")
    index = _device(logits, tokens, flags)
    if _elsewhere(index, stream):
        with _On(index, stream, (logits, tokens, flags)):
            return log_probs(logits, tokens, scale=scale, top_k=top_k, entropy=entropy, flags=flags)
    dev = logits.device
    # rows of one allocation: row_max, log_sum, logp, lse (, entropy)
    f = torch.empty((5 if entropy else 4, rows), dtype=torch.float32, device=dev)
    p, ids, alt, ids_p, alt_p = f.data_ptr(), None, None, None, None
    if top_k:
        ids = torch.empty((rows, top_k), dtype=torch.int32, device=dev)
        alt = torch.empty((rows, top_k), dtype=torch.float32, device=dev)
        ids_p, alt_p = ids.data_ptr(), alt.data_ptr()
    n = 4 * rows
    check(load_library().dobb_log_probs(
        logits.data_ptr(), dtype, rows, vocab, stride, tokens.data_ptr(), token_bytes, scale, top_k, p + 2 * n, p + 3 * n, p,
        p + n, p + 4 * n if entropy else None, ids_p, alt_p, _flags(flags), _raw_stream(index)))
    return LogProbs(f[2], f[3], f[4] if entropy else None, ids, alt, f, float(scale))


def log_probs_backward(logits: torch.Tensor, tokens: torch.Tensor, result: LogProbs, grad_logp: torch.Tensor, *,
                       grad_entropy: Optional[torch.Tensor] = None, grad_lse: Optional[torch.Tensor] = None,
                       out: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Gradient with respect to the logits, given `log_probs`' result on the
    same logits and tokens and the gradients of logp, of the entropy and of
    lse (float32, one per row).  `out` may be the logits themselves, or share no
    memory with them."""
    stride = _rows(logits, "logits")
    dtype = _float_dtype(logits.dtype, "logits")
    rows, vocab = logits.shape
    token_bytes = _token_bytes(tokens)
    if tokens.numel() != rows:
        raise ValueError(f"{tokens.numel()} tokens for {rows} rows")
    if grad_entropy is not None and result.entropy is None:
        raise ValueError("grad_entropy needs a result with the entropy")
    index = _device(logits, tokens, grad_logp, grad_entropy, grad_lse, out, result.stats)
    if _elsewhere(index, stream):
        with _On(index, stream, (logits, tokens, out, grad_logp, grad_entropy, grad_lse, result.stats,
                                 result.entropy)):
            return log_probs_backward(logits, tokens, result, grad_logp, grad_entropy=grad_entropy, grad_lse=grad_lse, out=out)
    stats = result.stats
    if stats.dtype != torch.float32 or not stats.is_contiguous() or stats.dim() != 2 or stats.shape[0] < 2 or stats.shape[1] != rows:
        raise ValueError(f"the result is not one for {rows} rows")
    args = [stats.data_ptr(), stats.data_ptr() + 4 * rows,
            _vector(result.entropy if grad_entropy is not None else None, rows, "entropy"),
            _vector(grad_logp, rows, "grad_logp"), _vector(grad_entropy, rows, "grad_entropy"),
            _vector(grad_lse, rows, "grad_lse")]
    if out is None:
        out = torch.empty((rows, vocab), dtype=logits.dtype, device=logits.device)
    elif out.shape != logits.shape or out.dtype != logits.dtype:
        raise ValueError("out must have the logits' shape and dtype")
    check(load_library().dobb_log_probs_backward(
        logits.data_ptr(), dtype, rows, vocab, stride, tokens.data_ptr(), token_bytes, result.scale, *args, out.data_ptr(),
        _rows(out, "out"), _raw_stream(index)))
    return out


# -------------------------------------------------------------------- embedding

def embedding(weight: torch.Tensor, tokens: torch.Tensor, *, scale: float = 1.0, out_dtype: Optional[torch.dtype] = None,
              out: Optional[torch.Tensor] = None, flags: Optional[torch.Tensor] = None,
              stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """scale * weight[tokens] as tokens.shape + (dim,), in out_dtype (default:
    the weight's).  Tokens below 0 are padding and give zeros.

    weight: (vocab, dim) float32 or bfloat16 with contiguous rows; `out`: a
    (tokens, dim) matrix with contiguous rows, apart from the weight."""
    wstride = _rows(weight, "weight")
    wdtype = _float_dtype(weight.dtype, "weight")
    vocab, dim = weight.shape
    token_bytes = _token_bytes(tokens)
    count = tokens.numel()
    if out is not None and out_dtype not in (None, out.dtype):
        raise ValueError(f"out has dtype {out.dtype}")
    odtype = _float_dtype(out.dtype if out is not None else (out_dtype or weight.dtype), "out dtype")
    index = _device(weight, tokens, out, flags)
    if _elsewhere(index, stream):
        with _On(index, stream, (weight, tokens, out, flags)):
            return embedding(weight, tokens, scale=scale, out_dtype=out_dtype, out=out, flags=flags)
    if out is None:
        out = torch.empty((*tokens.shape, dim), dtype=out_dtype or weight.dtype, device=weight.device)
        ostride = dim
    else:
        ostride = _rows(out, "out")
        if out.shape != (count, dim):
            raise ValueError(f"out must be {count} x {dim}")
    check(load_library().dobb_embedding(
        weight.data_ptr(), wdtype, vocab, dim, wstride, tokens.data_ptr(), token_bytes, count, scale, out.data_ptr(), odtype,
        ostride, _flags(flags), _raw_stream(index)))
    return out


def embedding_backward(grad: torch.Tensor, tokens: torch.Tensor, vocab: Optional[int] = None, *, scale: float = 1.0,
                       dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None, accumulate: bool = False,
                       flags: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Gradient of `embedding` with respect to the weight, (vocab, dim): the
    rows of `grad` of each token, times scale, summed in fp32.  Rows of tokens
    that do not occur are zero, or with `accumulate` stay as `out` has them.

    grad: tokens.shape + (dim,) contiguous, or a (tokens, dim) matrix with
    contiguous rows; `out`: (vocab, dim) with contiguous rows, apart from grad."""
    token_bytes = _token_bytes(tokens)
    count = tokens.numel()
    if grad.dim() < 1 or grad.numel() != count * grad.shape[-1]:
        raise ValueError(f"grad of shape {tuple(grad.shape)} for {count} tokens")
    dim = grad.shape[-1]
    if grad.dim() != 2:
        if not grad.is_contiguous():
            raise ValueError("grad must be contiguous, or a matrix")
        grad = grad.view(count, dim)
    if grad.shape[0] != count:
        raise ValueError(f"grad has {grad.shape[0]} rows for {count} tokens")
    gstride = _rows(grad, "grad")
    gdtype = _float_dtype(grad.dtype, "grad")
    if out is None:
        if accumulate or vocab is None:
            raise ValueError("accumulate needs out" if accumulate else "vocab or out must be given")
    else:
        if dtype not in (None, out.dtype):
            raise ValueError(f"out has dtype {out.dtype}")
        if out.dim() != 2 or out.shape[1] != dim or (vocab is not None and out.shape[0] != vocab):
            raise ValueError(f"out must be {'vocab' if vocab is None else vocab} x {dim}")
        vocab = out.shape[0]
    odtype = _float_dtype(out.dtype if out is not None else (dtype or grad.dtype), "out dtype")
    index = _device(grad, tokens, out, flags)
    if _elsewhere(index, stream):
        with _On(index, stream, (grad, tokens, out, flags)):
            return embedding_backward(grad, tokens, vocab, scale=scale, dtype=dtype, out=out, accumulate=accumulate, flags=flags)
    lib = load_library()
    nbytes = lib.dobb_embedding_backward_bytes(count, vocab, dim)
    if nbytes == 0:
        check(1)
    if out is None:
        out = torch.empty((vocab, dim), dtype=dtype or grad.dtype, device=grad.device)
    ws = torch.empty((nbytes,), dtype=torch.uint8, device=grad.device)
    check(lib.dobb_embedding_backward(
        grad.data_ptr(), gdtype, count, dim, gstride, tokens.data_ptr(), token_bytes, vocab, scale, out.data_ptr(), odtype,
        _rows(out, "out"), int(accumulate), _flags(flags), ws.data_ptr(), nbytes, _raw_stream(index)))
    return out


# --------------------------------------------------------------------- clipping

def _dense(t: torch.Tensor) -> bool:
    """Whether t's entries fill one stretch of memory, in any order of its dimensions."""
    if t.is_contiguous():
        return True
    need = 1
    for stride, size in sorted((st, sz) for sz, st in zip(t.shape, t.stride()) if sz > 1):
        if stride != need:
            return False
        need *= size
    return True


_dtype_of = attrgetter("dtype")


def _dtype_codes(tensors, what: str) -> array:
    kinds = set(map(_dtype_of, tensors))
    for d in kinds:
        if d not in _DTYPES:
            raise ValueError(f"every {what} must be float32 or bfloat16, got {d}")
    if len(kinds) == 1:
        return array("i", (_DTYPES[kinds.pop()],)) * len(tensors)
    return array("i", [_DTYPES[t.dtype] for t in tensors])


def _same_device(tensors, index: int) -> None:
    if set(map(torch.Tensor.get_device, tensors)) != {index}:
        raise ValueError(f"all tensors must be on cuda:{index}")


def _clip(grads: Sequence[torch.Tensor], max_norm: float, outs: Optional[Sequence[torch.Tensor]],
          flags: Optional[torch.Tensor], stream: Optional[torch.cuda.Stream]) -> GradNorm:
    n = len(grads)
    if n == 0:
        raise ValueError("no gradients given")
    in_place = outs is grads
    index = _device(grads[0], flags)
    _same_device(grads, index)
    gd = _dtype_codes(grads, "gradient")
    plain = all(map(torch.Tensor.is_contiguous, grads))
    if not plain and not all(map(_dense, grads)):
        raise ValueError("every gradient must be dense")
    ne = array("q", map(torch.Tensor.numel, grads))
    od = gd
    if outs is not None and not in_place:
        if len(outs) != n or array("q", map(torch.Tensor.numel, outs)) != ne:
            raise ValueError("there must be an output of the same size for every gradient")
        _same_device(outs, index)
        od = _dtype_codes(outs, "output")
        if not (plain and all(map(torch.Tensor.is_contiguous, outs))) and not all(
                (g.shape == o.shape and g.stride() == o.stride()) or (g.is_contiguous() and o.is_contiguous())
                for g, o in zip(grads, outs)):
            raise ValueError("every output must be laid out like its gradient")
    if _elsewhere(index, stream):
        with _On(index, stream, [*grads, *(outs or ()), flags]):
            return _clip(grads, max_norm, outs, flags, None)
    lib = load_library()
    gp = array("Q", map(torch.Tensor.data_ptr, grads))
    op = None if outs is None else gp if in_place else array("Q", map(torch.Tensor.data_ptr, outs))
    sizes = ne.buffer_info()[0]
    nbytes = lib.dobb_clip_grads_bytes(n, sizes)
    if nbytes == 0:
        check(1)
    # the statistics, and behind them the workspace, in one allocation
    at = (8 + 4 * n + 255) // 256 * 64
    stats = torch.empty((at + (nbytes + 3) // 4,), dtype=torch.float32, device=grads[0].device)
    p = stats.data_ptr()
    check(lib.dobb_clip_grads(
        n, gp.buffer_info()[0], gd.buffer_info()[0], sizes, max_norm, None if op is None else op.buffer_info()[0],
        None if op is None else od.buffer_info()[0], p, _flags(flags), p + 4 * at, nbytes, _raw_stream(index)))
    return GradNorm(stats[0], stats[1], stats[2:2 + n])


def grad_norm(grads: Sequence[torch.Tensor], *, flags: Optional[torch.Tensor] = None,
              stream: Optional[torch.cuda.Stream] = None) -> GradNorm:
    """The l2 norm over all entries of all gradients, and each tensor's own."""
    return _clip(list(grads), 0.0, None, flags, stream)


def clip_grads(grads: Sequence[torch.Tensor], max_norm: float, *, out: Optional[Sequence[torch.Tensor]] = None,
               flags: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> GradNorm:
    """Scale the gradients by min(1, max_norm / norm), norm the l2 norm over
    all of them: in place, or into `out` (as many entries each, laid out alike,
    float32 or bfloat16: for instance fp32 accumulators into the bf16 gradients that
    `Dobb.step` takes).  When the norm is not finite the gradients are passed
    on unscaled and flag 2 (non-finite gradient) is set in `flags`.

    grads: float32 or bfloat16 tensors, mixed if need be, of any shapes, none of
    them listed twice: no output may share memory with another tensor."""
    if not max_norm >= 0:
        raise ValueError(f"max_norm must be >= 0, got {max_norm}")
    grads = list(grads)
    return _clip(grads, float(max_norm), grads if out is None else list(out), flags, stream)
