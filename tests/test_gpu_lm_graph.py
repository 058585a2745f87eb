"""The operators inside a CUDA graph: nothing synchronises or allocates behind
the caller's back, so a captured call replays on new data in the same buffers."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_every_operator_replays_in_a_graph():
    import block_eigenbasis_preconditioning_gb300 as d
    gen = torch.Generator(device="cuda").manual_seed(3)
    R = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    vocab, dim, n = 3001, 96, 700
    logits, tokens, g = R(n, vocab), torch.randint(0, vocab, (n,), device="cuda", generator=gen), R(n)
    few, weight, grads = R(3, 40000), R(vocab, dim), R(n, dim)
    params = [R(300, 40), R(7), R(1000, 33)]
    outs = [torch.empty_like(p, dtype=torch.bfloat16) for p in params]
    tied = R(vocab, dim)

    def step():
        r = d.log_probs(logits, tokens, top_k=4)
        dl = d.log_probs_backward(logits, tokens, r, g, grad_entropy=g)
        q = d.log_probs(few, tokens[:3], top_k=2)
        e = d.embedding(weight, tokens, scale=2.0)
        dw = d.embedding_backward(grads, tokens, vocab)
        d.embedding_backward(grads, tokens, out=tied, accumulate=True)
        c = d.clip_grads(params, 0.5, out=outs)
        return [r.logp, r.entropy, r.top_ids, r.top_logp, dl, q.logp, q.top_ids, e, dw, tied, c.norm, c.norms, *outs]

    step()
    start = tied.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for _ in range(3):
        for t in (logits, g, few, weight, grads, *params):
            t.copy_(torch.randn(t.shape, device="cuda", generator=gen))
        tokens.copy_(torch.randint(0, vocab, (n,), device="cuda", generator=gen))
        tied.copy_(start)
        graph.replay()
        got = [t.clone() for t in captured]
        tied.copy_(start)
        for a, b in zip(got, step()):
            assert torch.equal(a, b)
