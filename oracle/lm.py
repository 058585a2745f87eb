"""Plain fp64 definitions of the language-model operators: log probabilities
and their gradient, the embedding lookup and its gradient, the global gradient
norm and clipping.

TEST INFRASTRUCTURE ONLY.  Row by row and entry by entry from the formulas
(the standard softmax, scatter-add and l2-norm definitions; the pages have no
counterpart); shares no code with the CUDA implementation.  Pinned in
tests/test_lm_oracle.py by hand-computed rows, finite differences and planted
mistakes.
"""
from __future__ import annotations

import math

import numpy as np

__all__ = ["log_probs", "log_probs_backward", "top_indices", "embedding", "embedding_backward",
           "clip_grads"]


def top_indices(x: np.ndarray, k: int) -> np.ndarray:
    """Indices of the k largest entries, largest first, ties by the lowest
    index; -0 equals 0 and a NaN is larger than every number."""
    nan = np.isnan(x)
    return np.lexsort((np.arange(len(x)), -np.where(nan, 0.0, x), ~nan))[:k]


def log_probs(logits: np.ndarray, tokens: np.ndarray, scale: float = 1.0, top_k: int = 0) -> dict:
    """logp, lse, entropy, row_max, log_sum (rows) and top_ids, top_logp (rows x top_k)."""
    rows = len(logits)
    r = {n: np.zeros(rows) for n in ("logp", "lse", "entropy", "row_max", "log_sum")}
    r["top_ids"] = np.zeros((rows, top_k), dtype=np.int64)
    r["top_logp"] = np.zeros((rows, top_k))
    for i in range(rows):
        x = logits[i].astype(np.float64)
        bad = bool(np.any(np.isnan(x)) or np.any(x == np.inf))
        m = float(np.max(x[~np.isnan(x)], initial=-np.inf))  # NaN are passed over
        if bad:
            log_sum = lse = ent = math.nan
            lp = np.full(len(x), math.nan)
        elif m == -np.inf:
            log_sum = lse = -math.inf
            ent = 0.0
            lp = np.full(len(x), -math.inf)
        else:
            e = np.exp(scale * (x - m))
            log_sum = math.log(e.sum())
            lse = scale * m + log_sum
            lp = scale * (x - m) - log_sum
            p = np.exp(lp)
            ent = -float((p[p > 0] * lp[p > 0]).sum())
        t = int(tokens[i])
        r["logp"][i] = 0.0 if t < 0 else (math.nan if t >= len(x) else lp[t])
        r["lse"][i], r["entropy"][i], r["row_max"][i], r["log_sum"][i] = lse, ent, m, log_sum
        r["top_ids"][i] = top_indices(x, top_k)
        r["top_logp"][i] = lp[r["top_ids"][i]]
    return r


def log_probs_backward(logits: np.ndarray, tokens: np.ndarray, grad_logp: np.ndarray, grad_entropy=None,
                       grad_lse=None, scale: float = 1.0) -> np.ndarray:
    """d/d logits of sum(grad_logp logp + grad_entropy entropy + grad_lse lse)."""
    d = np.zeros(logits.shape)
    f = log_probs(logits, tokens, scale)
    for i in range(len(logits)):
        if f["log_sum"][i] == -math.inf:
            continue
        lp = scale * (logits[i].astype(np.float64) - f["row_max"][i]) - f["log_sum"][i]
        p = np.exp(lp)
        t = int(tokens[i])
        given = 0 <= t < logits.shape[1]
        g = float(grad_logp[i]) if given else 0.0
        h = 0.0 if grad_entropy is None else float(grad_entropy[i])
        l = 0.0 if grad_lse is None else float(grad_lse[i])
        plogp = np.where(p > 0, p * np.where(p > 0, lp, 0.0), 0.0) if not math.isnan(f["log_sum"][i]) else p
        d[i] = (l - g) * p - h * (plogp + p * f["entropy"][i])
        if given:
            d[i, t] += g
    return scale * d


def embedding(weight: np.ndarray, tokens: np.ndarray, scale: float = 1.0) -> np.ndarray:
    out = np.zeros((len(tokens), weight.shape[1]))
    for i, t in enumerate(tokens):
        if 0 <= t < len(weight):
            out[i] = scale * weight[t].astype(np.float64)
    return out


def embedding_backward(grad: np.ndarray, tokens: np.ndarray, vocab: int, scale: float = 1.0, add_to=None):
    """(dweight, the sum of the absolute values that went into each entry)."""
    d = np.zeros((vocab, grad.shape[1]))
    a = np.zeros_like(d)
    if add_to is not None:
        d += add_to
        a += np.abs(add_to)
    for i, t in enumerate(tokens):
        if 0 <= t < vocab:
            d[t] += scale * grad[i].astype(np.float64)
            a[t] += abs(scale) * np.abs(grad[i].astype(np.float64))
    return d, a


def clip_grads(grads, max_norm: float):
    """(norm, factor, norms, scaled gradients)."""
    with np.errstate(over="ignore", invalid="ignore"):
        norms = np.array([math.sqrt(float((g.astype(np.float64).ravel() ** 2).sum())) for g in grads])
        norm = math.sqrt(float((norms ** 2).sum()))
    c = max_norm / norm if math.isfinite(norm) and norm > max_norm else 1.0
    return norm, c, norms, [c * g.astype(np.float64) for g in grads]
