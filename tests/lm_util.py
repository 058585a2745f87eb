"""Shared helpers of the GPU tests of the language-model operators: inputs on
the device and error bounds of a 32-bit evaluation, derived before any run.

u = 2^-24 is half the spacing of fp32 around 1.  The bounds hold for any
order of summation whose chains are at most `chain` additions long:

* log probabilities, w_j = scale (x_j - max): w_j has two roundings, the
  exponential a few units, so e^{w_j} is off by at most (2 |w_j| + 8) u of
  itself, and the sum S by (2 W + 8 + chain) u, W = sum_j p_j |w_j| (a mean of
  the |w_j|).  log S is off by that, plus its own rounding u |log S| (2 more
  for the logarithm's units); logp = w_t - log S adds 2 u |w_t| and one
  rounding.
* entropy = log S - E / S with E = sum e^{w_j} w_j: every term is off by
  (2 |w_j| + 10) u of itself, the sum by chain more, so E / S is off by at most
  u (2 sum p_j w_j^2 + (10 + chain) W) plus W times the error of S.
* gradients: from the errors of log p_j and of the entropy, see grad_bound.
* a result of fewer bits adds half a unit of its type: bf16 has 8 significant
  bits, so numbers in [1, 2) are 2^-7 apart and rounding moves them by up to
  2^-8.
"""
from __future__ import annotations

import numpy as np
import torch

U = 2.0 ** -24
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF_UNIT = {"f32": U, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133}  # spacing of the subnormals


def chain(vocab: int) -> int:
    """Longest chain of additions over a row: vocab entries over at least 128
    threads of a block, then joins of at most 64 parts."""
    return vocab // 128 + 64


def stats_bounds(logits: np.ndarray, scale: float, f: dict):
    """Per row: error bounds of log_sum and of the entropy, for finite rows."""
    eS, eH = np.zeros(len(logits)), np.zeros(len(logits))
    n = chain(logits.shape[1])
    for i, x in enumerate(logits.astype(np.float64)):
        if not np.isfinite(f["log_sum"][i]):
            continue
        w = scale * (x[np.isfinite(x)] - f["row_max"][i])
        p = np.exp(w - f["log_sum"][i])
        W, W2 = float((p * -w).sum()), float((p * w * w).sum())
        rel = U * (2 * W + 8 + n)
        eS[i] = rel + 3 * U * abs(f["log_sum"][i]) + U
        eH[i] = eS[i] + U * (2 * W2 + (10 + n) * W) + W * rel + 3 * U * (W + abs(f["log_sum"][i]))
    return eS, eH


def logp_bound(w: np.ndarray, log_sum: np.ndarray, eS: np.ndarray) -> np.ndarray:
    """Bound of w - log_sum, w = scale (x - max)."""
    return eS + U * (4 * np.abs(w) + 2 * np.abs(log_sum)) + U


def grad_bound(logits, tokens, f, eS, eH, g, h, l, scale, dtype) -> np.ndarray:
    """Per entry bound of the gradient: with lp = log p_j off by e, p is off by
    p (e + 8 u); the factor (l - g - h (lp + H)) by |h| (e + eH) and its own
    few roundings."""
    b = np.zeros(logits.shape)
    for i, x in enumerate(logits.astype(np.float64)):
        if not np.isfinite(f["log_sum"][i]):
            continue
        w = np.where(np.isfinite(x), scale * (x - f["row_max"][i]), -1e4)
        lp = w - f["log_sum"][i]
        p = np.exp(lp)
        e = logp_bound(w, f["log_sum"][i], eS[i])
        hh = 0.0 if h is None else abs(float(h[i]))
        size = abs(float(g[i])) + (0.0 if l is None else abs(float(l[i]))) + hh * (np.abs(lp) + abs(f["entropy"][i]))
        b[i] = p * (size * (e + 16 * U) + hh * (e + eH[i]))
        t = int(tokens[i])
        if 0 <= t < logits.shape[1]:
            b[i, t] += 4 * U * abs(float(g[i]))
        b[i] += 2 * U * p * size
    return b * scale


def dev(x: np.ndarray, dtype: str) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).cuda().to(TORCH[dtype])


def np64(t: torch.Tensor) -> np.ndarray:
    return t.detach().double().cpu().numpy()


def rounded(x: np.ndarray, dtype: str) -> np.ndarray:
    """The values that the type holds, in fp32."""
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(TORCH[dtype]).float().numpy()


def strided(x: np.ndarray, dtype: str, extra: int = 0, offset: int = 0) -> torch.Tensor:
    """x on the device as a matrix with `extra` columns between its rows (NaN,
    so that a read past a row shows) and `offset` elements before it."""
    rows, cols = x.shape
    buf = torch.full((offset + rows * (cols + extra) + 8,), float("nan"), dtype=TORCH[dtype], device="cuda")
    v = buf[offset:offset + rows * (cols + extra)].view(rows, cols + extra)[:, :cols]
    v.copy_(dev(x, dtype))
    return v


def assert_close(got: np.ndarray, want: np.ndarray, bound, what: str = "") -> None:
    """Non-finite entries equal, finite ones within the bound; what lies beyond
    the range of fp32 reads as an infinity."""
    want = np.where(np.abs(want) > np.finfo(np.float32).max, np.sign(want) * np.inf, want)
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), what
    assert np.array_equal(got[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)]), what
    b = np.broadcast_to(bound, want.shape)[fine]
    err = np.abs(got[fine] - want[fine])
    assert np.isfinite(got[fine]).all() and (err <= b).all(), \
        f"{what}: worst error {float((err - b).max()) if err.size else 0:.3g} above its bound, {float(err.max()):.3g} in all"
