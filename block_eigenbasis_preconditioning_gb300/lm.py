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
Wrong arguments raise ValueError before anything is launched.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional, Sequence

import torch

from .binding import check, load_library

_DTYPES = {torch.float32: 0, torch.bfloat16: 1}
_TOKEN_BYTES = {torch.int32: 4, torch.int64: 8}
MAX_TOP_K = 32


class LogProbs(NamedTuple):
    """Result of `log_probs`, one entry per row (the alternatives: one row of
    top_k).  row_max, log_sum and scale are what `log_probs_backward` needs:
    lse = scale * row_max + log_sum."""
    logp: torch.Tensor
    lse: torch.Tensor
    entropy: Optional[torch.Tensor]
    top_ids: Optional[torch.Tensor]
    top_logp: Optional[torch.Tensor]
    row_max: torch.Tensor
    log_sum: torch.Tensor
    scale: float


class GradNorm(NamedTuple):
    """Result of `grad_norm` and `clip_grads`: the global norm, the factor the
    gradients were multiplied with, and every tensor's own norm, fp32 on the
    device."""
    norm: torch.Tensor
    scale: torch.Tensor
    norms: torch.Tensor


def _need(ok: bool, msg: str, *args) -> None:
    if not ok:
        raise ValueError(msg.format(*args))


def _device_of(first: torch.Tensor, *others: Optional[torch.Tensor]) -> torch.device:
    dev = first.device
    _need(dev.type == "cuda", "tensors must be on a CUDA device, got {}", dev)
    for t in others:
        _need(t is None or t.device == dev, "all tensors must be on {}", dev)
    return dev


def _rows(t: torch.Tensor, name: str) -> int:
    """Row stride of a matrix whose rows are contiguous."""
    _need(t.dim() == 2, "{} must be a matrix, got {} dimensions", name, t.dim())
    _need(t.stride(1) == 1 or t.shape[1] <= 1, "{} must have contiguous rows", name)
    _need(t.stride(0) >= t.shape[1] or t.shape[0] <= 1, "{} must not overlap itself", name)
    return max(t.stride(0), t.shape[1])


def _tokens(t: torch.Tensor, name: str) -> int:
    _need(t.dtype in _TOKEN_BYTES, "{} must be int32 or int64, got {}", name, t.dtype)
    _need(t.is_contiguous(), "{} must be contiguous", name)
    return _TOKEN_BYTES[t.dtype]


def _vector(t: Optional[torch.Tensor], n: int, name: str) -> Optional[int]:
    if t is None:
        return None
    _need(t.dtype == torch.float32 and t.is_contiguous() and t.numel() == n,
          "{} must be {} contiguous float32 values", name, n)
    return t.data_ptr()


def _flags(flags: Optional[torch.Tensor]) -> Optional[int]:
    if flags is None:
        return None
    _need(flags.dtype in (torch.int32, torch.uint32) and flags.numel() == 1,
          "flags must be one int32 or uint32")
    return flags.data_ptr()


def _float_dtype(dtype: torch.dtype, name: str) -> int:
    _need(dtype in _DTYPES, "{} must be float32 or bfloat16, got {}", name, dtype)
    return _DTYPES[dtype]


class _On:
    """The device and stream of a call: allocations inside come from that
    stream, and inputs made on another stream outlive the work on it."""

    def __init__(self, device: torch.device, stream: Optional[torch.cuda.Stream], used):
        self.ctx = []
        if stream is not None and stream != torch.cuda.current_stream(device):
            _need(stream.device == device, "the stream is on {}, the tensors on {}", stream.device, device)
            self.ctx.append(torch.cuda.stream(stream))
            for t in used:
                if t is not None:
                    t.record_stream(stream)
        elif device.index != torch.cuda.current_device():
            self.ctx.append(torch.cuda.device(device))
        self.ptr = (stream if stream is not None else torch.cuda.current_stream(device)).cuda_stream

    def __enter__(self):
        for c in self.ctx:
            c.__enter__()
        return self.ptr

    def __exit__(self, *exc):
        for c in reversed(self.ctx):
            c.__exit__(*exc)


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
    token_bytes = _tokens(tokens, "tokens")
    _need(tokens.numel() == rows, "{} tokens for {} rows", tokens.numel(), rows)
    _need(0 <= top_k <= min(MAX_TOP_K, vocab), "top_k must lie in [0, min({}, vocab)], got {}", MAX_TOP_K, top_k)
    dev = _device_of(logits, tokens, flags)
    lib = load_library()
    with _On(dev, stream, (logits, tokens, flags)) as s:
        f = torch.empty(5 if entropy else 4, rows, dtype=torch.float32, device=dev)
        ids = torch.empty(rows, top_k, dtype=torch.int32, device=dev) if top_k else None
        alt = torch.empty(rows, top_k, dtype=torch.float32, device=dev) if top_k else None
        p = f.data_ptr()
        check(lib.dobb_log_probs(
            logits.data_ptr(), dtype, rows, vocab, stride, tokens.data_ptr(), token_bytes, scale, top_k, p, p + 4 * rows,
            p + 8 * rows, p + 12 * rows, p + 16 * rows if entropy else None, ids.data_ptr() if top_k else None,
            alt.data_ptr() if top_k else None, _flags(flags), s))
    return LogProbs(f[0], f[1], f[4] if entropy else None, ids, alt, f[2], f[3], float(scale))


def log_probs_backward(logits: torch.Tensor, tokens: torch.Tensor, result: LogProbs, grad_logp: torch.Tensor, *,
                       grad_entropy: Optional[torch.Tensor] = None, grad_lse: Optional[torch.Tensor] = None,
                       out: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Gradient with respect to the logits, given `log_probs`' result on the
    same logits and tokens and the gradients of logp, of the entropy and of
    lse (float32, one per row).  `out` may be the logits themselves."""
    stride = _rows(logits, "logits")
    dtype = _float_dtype(logits.dtype, "logits")
    rows, vocab = logits.shape
    token_bytes = _tokens(tokens, "tokens")
    _need(tokens.numel() == rows, "{} tokens for {} rows", tokens.numel(), rows)
    _need(grad_entropy is None or result.entropy is not None, "grad_entropy needs a result with the entropy")
    dev = _device_of(logits, tokens, grad_logp, grad_entropy, grad_lse, out, result.row_max)
    args = [_vector(result.row_max, rows, "row_max"), _vector(result.log_sum, rows, "log_sum"),
            _vector(result.entropy if grad_entropy is not None else None, rows, "entropy"),
            _vector(grad_logp, rows, "grad_logp"), _vector(grad_entropy, rows, "grad_entropy"),
            _vector(grad_lse, rows, "grad_lse")]
    lib = load_library()
    with _On(dev, stream, (logits, tokens, out, grad_logp, grad_entropy, grad_lse, result.row_max, result.log_sum,
                           result.entropy)) as s:
        if out is None:
            out = torch.empty(rows, vocab, dtype=logits.dtype, device=dev)
        _need(out.shape == logits.shape and out.dtype == logits.dtype, "out must have the logits' shape and dtype")
        check(lib.dobb_log_probs_backward(logits.data_ptr(), dtype, rows, vocab, stride, tokens.data_ptr(), token_bytes,
                                          result.scale, *args, out.data_ptr(), _rows(out, "out"), s))
    return out


# -------------------------------------------------------------------- embedding

def embedding(weight: torch.Tensor, tokens: torch.Tensor, *, scale: float = 1.0, out_dtype: Optional[torch.dtype] = None,
              out: Optional[torch.Tensor] = None, flags: Optional[torch.Tensor] = None,
              stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """scale * weight[tokens] as tokens.shape + (dim,), in out_dtype (default:
    the weight's).  Tokens below 0 are padding and give zeros.

    weight: (vocab, dim) float32 or bfloat16 with contiguous rows; `out`: a
    (tokens, dim) matrix with contiguous rows."""
    wstride = _rows(weight, "weight")
    wdtype = _float_dtype(weight.dtype, "weight")
    vocab, dim = weight.shape
    token_bytes = _tokens(tokens, "tokens")
    count = tokens.numel()
    _need(out is None or out_dtype in (None, out.dtype), "out has dtype {}", out.dtype if out is not None else None)
    odtype = _float_dtype(out.dtype if out is not None else (out_dtype or weight.dtype), "out dtype")
    dev = _device_of(weight, tokens, out, flags)
    lib = load_library()
    with _On(dev, stream, (weight, tokens, out, flags)) as s:
        if out is None:
            out = torch.empty(tokens.shape + (dim,), dtype=out_dtype or weight.dtype, device=dev)
            ostride = dim
        else:
            ostride = _rows(out, "out")
            _need(tuple(out.shape) == (count, dim), "out must be {} x {}", count, dim)
        check(lib.dobb_embedding(weight.data_ptr(), wdtype, vocab, dim, wstride, tokens.data_ptr(), token_bytes, count, scale,
                                 out.data_ptr(), odtype, ostride, _flags(flags), s))
    return out


def embedding_backward(grad: torch.Tensor, tokens: torch.Tensor, vocab: Optional[int] = None, *, scale: float = 1.0,
                       dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None, accumulate: bool = False,
                       flags: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Gradient of `embedding` with respect to the weight, (vocab, dim): the
    rows of `grad` of each token, times scale, summed in fp32.  Rows of tokens
    that do not occur are zero, or with `accumulate` stay as `out` has them.

    grad: tokens.shape + (dim,) contiguous, or a (tokens, dim) matrix with
    contiguous rows; `out`: (vocab, dim) with contiguous rows."""
    token_bytes = _tokens(tokens, "tokens")
    count = tokens.numel()
    _need(grad.dim() >= 1, "grad must have a last dimension")
    dim = grad.shape[-1]
    _need(grad.numel() == count * dim, "grad has {} values for {} tokens of {}", grad.numel(), count, dim)
    if grad.dim() != 2:
        _need(grad.is_contiguous(), "grad must be contiguous, or a matrix")
        grad = grad.view(count, dim)
    _need(grad.shape[0] == count, "grad has {} rows for {} tokens", grad.shape[0], count)
    gstride = _rows(grad, "grad")
    gdtype = _float_dtype(grad.dtype, "grad")
    _need(out is not None or not accumulate, "accumulate needs out")
    _need(out is not None or vocab is not None, "vocab or out must be given")
    _need(out is None or dtype in (None, out.dtype), "out has dtype {}", out.dtype if out is not None else None)
    dev = _device_of(grad, tokens, out, flags)
    lib = load_library()
    with _On(dev, stream, (grad, tokens, out, flags)) as s:
        if out is None:
            out = torch.empty(int(vocab), dim, dtype=dtype or grad.dtype, device=dev)
        _need(out.dim() == 2 and out.shape[1] == dim and (vocab is None or out.shape[0] == vocab),
              "out must be {} x {}", vocab if vocab is not None else "vocab", dim)
        odtype = _float_dtype(out.dtype, "out dtype")
        nbytes = lib.dobb_embedding_backward_bytes(count, out.shape[0], dim)
        if nbytes == 0:
            check(1)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        check(lib.dobb_embedding_backward(grad.data_ptr(), gdtype, count, dim, gstride, tokens.data_ptr(), token_bytes,
                                          out.shape[0], scale, out.data_ptr(), odtype, _rows(out, "out"), int(accumulate),
                                          _flags(flags), ws.data_ptr(), nbytes, s))
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


def _clip(grads: Sequence[torch.Tensor], max_norm: float, outs: Optional[Sequence[torch.Tensor]],
          flags: Optional[torch.Tensor], stream: Optional[torch.cuda.Stream]) -> GradNorm:
    grads = list(grads)
    n = len(grads)
    _need(n > 0, "no gradients given")
    _need(outs is None or len(outs) == n, "{} outputs for {} gradients", 0 if outs is None else len(outs), n)
    dev = _device_of(*grads, flags)
    for i, g in enumerate(grads):
        _need(g.dtype in _DTYPES, "gradient {} must be float32 or bfloat16, got {}", i, g.dtype)
        _need(_dense(g), "gradient {} must be dense", i)
    if outs is not None and outs is not grads:
        _device_of(grads[0], *outs)
        for i, (g, o) in enumerate(zip(grads, outs)):
            _need(o.dtype in _DTYPES, "output {} must be float32 or bfloat16, got {}", i, o.dtype)
            _need(o.shape == g.shape and (o.stride() == g.stride() or (o.is_contiguous() and g.is_contiguous())),
                  "output {} must have its gradient's shape and strides", i)
    lib = load_library()
    gp = (ctypes.c_void_p * n)(*[g.data_ptr() for g in grads])
    gd = (ctypes.c_int32 * n)(*[_DTYPES[g.dtype] for g in grads])
    ne = (ctypes.c_int64 * n)(*[g.numel() for g in grads])
    op = od = None
    if outs is not None:
        op = (ctypes.c_void_p * n)(*[o.data_ptr() for o in outs])
        od = (ctypes.c_int32 * n)(*[_DTYPES[o.dtype] for o in outs])
    nbytes = lib.dobb_clip_grads_bytes(n, ne)
    if nbytes == 0:
        check(1)
    with _On(dev, stream, [*grads, *(outs or ()), flags]) as s:
        stats = torch.empty(2 + n, dtype=torch.float32, device=dev)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        check(lib.dobb_clip_grads(n, gp, gd, ne, max_norm, op, od, stats.data_ptr(), _flags(flags), ws.data_ptr(), nbytes, s))
    return GradNorm(stats[0], stats[1], stats[2:])


def grad_norm(grads: Sequence[torch.Tensor], *, flags: Optional[torch.Tensor] = None,
              stream: Optional[torch.cuda.Stream] = None) -> GradNorm:
    """The l2 norm over all entries of all gradients, and each tensor's own."""
    return _clip(grads, 0.0, None, flags, stream)


def clip_grads(grads: Sequence[torch.Tensor], max_norm: float, *, out: Optional[Sequence[torch.Tensor]] = None,
               flags: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> GradNorm:
    """Scale the gradients by min(1, max_norm / norm), norm the l2 norm over
    all of them: in place, or into `out` (same shapes, float32 or bfloat16
    each: for instance fp32 accumulators into the bf16 gradients that
    `Dobb.step` takes).  When the norm is not finite the gradients are passed
    on unscaled and flag 2 (non-finite gradient) is set in `flags`.

    grads: float32 or bfloat16 tensors, mixed if need be, of any shapes."""
    _need(max_norm >= 0, "max_norm must be >= 0, got {}", max_norm)
    grads = list(grads)
    return _clip(grads, float(max_norm), grads if out is None else list(out), flags, stream)
