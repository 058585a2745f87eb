"""A language model with a tied embedding, trained with Dobb.

    python examples/tied_lm.py [--steps 60]

One step, from the tokens to the new weights:

  embedding            x = scale * E[tokens]                     (lookup)
  (torch)              h = x W^T, logits = h E^T
  log_probs            log p(next token), its entropy
  log_probs_backward   gradient of  -mean(log p) - 0.01 mean(entropy)
  (torch)              the products' gradients, fp32
  embedding_backward   the lookup's gradient added onto the head's: E is tied
  clip_grads           global norm at most 1, fp32 accumulators -> bf16
  Dobb                 moments of the inputs (h of E, x of W), refresh, update

The data are a noisy walk over the vocabulary: the next token is a fixed
function of the last one four times out of five, anything otherwise.
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import block_eigenbasis_preconditioning_gb300 as dobb  # noqa: E402

ENTROPY_WEIGHT = 0.01


def batch(tokens: int, vocab: int, gen: torch.Generator):
    """tokens pairs (token, next token) of the walk."""
    cur = torch.randint(0, vocab, (tokens,), device="cuda", generator=gen)
    other = torch.randint(0, vocab, (tokens,), device="cuda", generator=gen)
    follow = torch.rand(tokens, device="cuda", generator=gen) < 0.8
    return cur, torch.where(follow, (7 * cur + 3) % vocab, other)


def loss_and_gradients(E: torch.Tensor, W: torch.Tensor, cur: torch.Tensor, nxt: torch.Tensor):
    """(loss, dE, dW in fp32, inputs of E's and of W's product)."""
    n, scale = cur.numel(), math.sqrt(E.shape[1])
    x = dobb.embedding(E, cur, scale=scale)
    h = x @ W.t()
    logits = h @ E.t()
    r = dobb.log_probs(logits, nxt)
    loss = -r.logp.mean() - ENTROPY_WEIGHT * r.entropy.mean()
    g = torch.full((n,), -1.0 / n, device=E.device)
    dlogits = dobb.log_probs_backward(logits, nxt, r, g, grad_entropy=ENTROPY_WEIGHT * g, out=logits)
    dh = dlogits @ E
    dE = (dlogits.t() @ h).float()
    dW = (dh.t() @ x).float()
    dobb.embedding_backward(dh @ W, cur, scale=scale, out=dE, accumulate=True)
    return loss, dE, dW, h, x


def train(steps: int = 60, tokens: int = 4096, vocab: int = 1000, dim: int = 128, lr: float = 3e-3, seed: int = 0):
    """Losses and gradient norms of the steps, and the model (E, W)."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    E = (torch.randn(vocab, dim, device="cuda", generator=gen) * 0.05).bfloat16()
    W = (torch.randn(dim, dim, device="cuda", generator=gen) / math.sqrt(dim)).bfloat16()
    opt = dobb.Dobb([(vocab, dim), (dim, dim)], B=4, refresh_period=10, param_dtype="bf16", act_dtype="bf16")
    G = [torch.empty_like(E), torch.empty_like(W)]
    losses, norms = [], []
    for _ in range(steps):
        cur, nxt = batch(tokens, vocab, gen)
        loss, dE, dW, h, x = loss_and_gradients(E, W, cur, nxt)
        clipped = dobb.clip_grads([dE, dW], 1.0, out=G)
        opt.accumulate([h, x])
        opt.step([E, W], G, lr)
        losses.append(loss)
        norms.append(clipped.norm)
    return torch.stack(losses).tolist(), torch.stack(norms).tolist(), (E, W)


def continue_from(E: torch.Tensor, W: torch.Tensor, token: int, top_k: int = 3):
    """The most likely next tokens and their probabilities."""
    cur = torch.tensor([token], device="cuda")
    logits = (dobb.embedding(E, cur, scale=math.sqrt(E.shape[1])) @ W.t()) @ E.t()
    r = dobb.log_probs(logits, torch.tensor([-1], device="cuda"), top_k=top_k)
    return r.top_ids[0].tolist(), r.top_logp[0].exp().tolist()


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=60)
    a = ap.parse_args()
    losses, norms, (E, W) = train(a.steps)
    for i in sorted({0, *range(9, a.steps, 10), a.steps - 1}):
        print(f"step {i + 1:4d}  loss {losses[i]:.4f}  gradient norm {norms[i]:.4f}")
    ids, p = continue_from(E, W, 5)
    print("after token 5:", ", ".join(f"{t} ({q:.2f})" for t, q in zip(ids, p)), f"(the walk goes to {7 * 5 + 3})")


if __name__ == "__main__":
    main()
