"""The operators at the two ends of a language model and on its gradients, as workloads to measure.

Three operators: log probabilities of given tokens (with entropy, the top alternatives and the
gradient), the token embedding (lookup and gradient), and gradient clipping by the global norm.
`run` with `own` false computes them from elementary torch operations in 32 bits; with `own` true it
makes the calls of this framework.  `exact` is the definition in 64 bits.

Definitions, y = scale * logits:
  lse = log sum_j exp(y_j); logp = y_t - lse; entropy = -sum_j p_j log p_j, p_j = exp(y_j - lse); the
  alternatives are the k largest logits, ties to the lowest index.  A row of -inf alone has lse = -inf,
  logp = -inf, entropy 0 and no gradient.  A token below 0 stands for none: logp 0.
  d logits_j = scale * (g (1[j = t] - p_j) - h p_j (log p_j + entropy)) for the gradients g of logp and
  h of the entropy.
  lookup: out[t] = scale * weight[id_t], zeros for an id below 0; its gradient
  d weight[v] = scale * sum of the rows t with id_t = v, optionally added to what is there.
  clip: norm = sqrt(sum of squares over all tensors); out = gradients * min(1, max_norm / norm).
"""
import math

import numpy as np
import torch

own = False

_DEV = "cuda" if torch.cuda.is_available() else "cpu"
_T = {"bf16": torch.bfloat16, "f32": torch.float32}
_INF = float("inf")


# ---------------------------------------------------------------------------------------- cases

def _logp(name, rows, vocab, dtype, top, entropy=True, grad=False, stride=0, banned=0.0, ragged=False, scale=1.0):
    return {"name": name, "op": "logp", "rows": rows, "vocab": vocab, "dtype": dtype, "top": top, "entropy": entropy, "grad": grad,
            "stride": stride or vocab, "banned": banned, "ragged": ragged, "scale": scale}


def _embed(name, tokens, vocab, dim, weight, out, scale=1.0, padded=0.0):
    return {"name": name, "op": "embed", "tokens": tokens, "vocab": vocab, "dim": dim, "weight": weight, "out": out, "scale": scale, "padded": padded}


def _embed_grad(name, tokens, vocab, dim, grad, weight, add, scale=1.0, padded=0.0):
    return {"name": name, "op": "embed_grad", "tokens": tokens, "vocab": vocab, "dim": dim, "grad": grad, "weight": weight, "add": add,
            "scale": scale, "padded": padded}


def _clip(name, layers, dim, ff, vocab, vectors, grad, out, max_norm):
    return {"name": name, "op": "clip", "layers": layers, "dim": dim, "ff": ff, "vocab": vocab, "vectors": vectors, "grad": grad, "out": out,
            "max_norm": max_norm}


def listed():
    return [
        # one sequence generating: the token's log probability and the five alternatives shown beside it
        _logp("logp-1x50257-bf16", 1, 50257, "bf16", 5, entropy=False),
        # a serving batch at a temperature, with the alternatives of an API answer, from 32-bit logits
        _logp("logp-64x128256-f32", 64, 128256, "f32", 20, scale=1.25),
        # scoring the 8192 tokens of the GPT-2 XL workload
        _logp("logp-8192x50257-bf16", 8192, 50257, "bf16", 5),
        # an odd batch with banned tokens, padded positions, rows where every token is banned, and a vocabulary padded to 50304 columns
        _logp("logp-1021x50257-f32-masked", 1021, 50257, "f32", 8, stride=50304, banned=0.3, ragged=True),
        # a training step's loss at the head: log probabilities, entropy and the gradient of both
        _logp("logp-train-8192x50257-bf16", 8192, 50257, "bf16", 0, grad=True),
        # the lookup of eight sequences generating
        _embed("embed-8x1600-bf16", 8, 50257, 1600, "bf16", "bf16"),
        # prompts of a Llama-3-8B batch from 32-bit weights, scaled by sqrt(d), some positions padded
        _embed("embed-16384x4096-f32-bf16", 16384, 128256, 4096, "f32", "bf16", scale=64.0, padded=0.1),
        # the GPT-2 XL embedding's gradient for 8192 tokens: all of 50257 x 1600 is written
        _embed_grad("embed-grad-8192x1600-bf16", 8192, 50257, 1600, "bf16", "bf16", False),
        # the same kind of gradient added onto the 32-bit gradient of a tied head, odd sizes
        _embed_grad("embed-grad-add-32761x1601", 32761, 50257, 1601, "bf16", "f32", True, scale=1.5, padded=0.1),
        # one 768 x 768 matrix, as in the framework's single-matrix workload
        _clip("clip-768x768-f32", 0, 768, 0, 768, False, "f32", "f32", 0.1),
        # GPT-2 Small's 72 matrices with its gains and biases
        _clip("clip-gpt2-small-f32", 12, 768, 3072, 0, True, "f32", "f32", 1.0),
        # GPT-2 XL: 289 matrices, 32-bit accumulated gradients to the 16 bits that the step takes
        _clip("clip-gpt2-xl-f32-bf16", 48, 1600, 6400, 50257, False, "f32", "bf16", 1.0),
    ]


def _size(rng, lo, hi):
    """A whole number spread over [lo, hi] by its logarithm."""
    while True:
        v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        if lo <= v <= hi and v != 3072:
            return v


def draw(rng):
    op = rng.choice(["logp", "logp", "embed", "embed_grad", "clip"])
    dtype = rng.choice(["bf16", "f32"])
    if op == "logp":
        vocab = rng.choice([50257, 128256, _size(rng, 1000, 131072), _size(rng, 1000, 131072)])
        rows = _size(rng, 1, min(8192, 8192 * 50257 // vocab))
        grad = rng.random() < 0.5
        c = _logp("", rows, vocab, dtype, 0 if grad else rng.randint(0, 20), entropy=grad or rng.random() < 0.5, grad=grad,
                  stride=vocab + rng.choice([0, 0, 1, 47]), banned=rng.choice([0.0, 0.0, 0.2]), ragged=rng.random() < 0.3,
                  scale=rng.choice([1.0, 0.7, 1.25]))
    elif op == "embed":
        vocab, dim = _size(rng, 1000, 131072), _size(rng, 64, 4096)
        c = _embed("", _size(rng, 1, 16384), vocab, dim, dtype, rng.choice(["bf16", "f32"]), scale=rng.choice([1.0, math.sqrt(dim)]),
                   padded=rng.choice([0.0, 0.2]))
    elif op == "embed_grad":
        c = _embed_grad("", _size(rng, 1, 32768), _size(rng, 1000, 131072), _size(rng, 64, 2048), dtype, rng.choice(["bf16", "f32"]),
                        rng.random() < 0.5, scale=rng.choice([1.0, 1.5]), padded=rng.choice([0.0, 0.2]))
    else:
        dim = _size(rng, 64, 1600)
        c = _clip("", rng.randint(0, 24), dim, _size(rng, dim, 4 * dim), _size(rng, 256, 50257), rng.random() < 0.5, dtype,
                  rng.choice(["bf16", "f32"]), rng.choice([0.01, 1.0]))
    del c["name"]
    return c


# --------------------------------------------------------------------------------------- inputs

def _generator(seed):
    return torch.Generator(device=_DEV).manual_seed(seed)


def _word_probs(vocab):
    """Token frequencies that fall with the rank, as in text; low ids are the frequent ones."""
    p = 1.0 / (np.arange(vocab, dtype=np.float64) + 2.7)
    return p / p.sum()


def _ids(tokens, vocab, padded, gen):
    cdf = torch.from_numpy(np.cumsum(_word_probs(vocab))).to(_DEV)
    ids = torch.searchsorted(cdf, torch.rand(tokens, device=_DEV, generator=gen, dtype=torch.float64)).clamp_(max=vocab - 1)
    if padded:
        ids[torch.rand(tokens, device=_DEV, generator=gen) < padded] = -1
    return ids


def _matrices(case):
    d, ff = case["dim"], case["ff"]
    layer = [(d, d)] * 4 + [(ff, d), (d, ff)]
    return layer * case["layers"] + ([(case["vocab"], d)] if case["vocab"] else [])


def _vectors(case):
    return [(case["dim"],)] * 8 * case["layers"] if case["vectors"] else []


def _flat(shapes, dtype):
    """A flat buffer and a view of it for each shape, each at a multiple of 64 values."""
    at = np.cumsum([0] + [(math.prod(s) + 63) // 64 * 64 for s in shapes]).tolist()
    flat = torch.zeros(at[-1], dtype=_T[dtype], device=_DEV)
    return flat, [flat[o:o + math.prod(s)].view(s) for o, s in zip(at, shapes)]


def prepare(case, seed):
    gen = _generator(seed)
    randn = lambda *s: torch.randn(*s, device=_DEV, generator=gen)  # noqa: E731
    rand = lambda *s: torch.rand(*s, device=_DEV, generator=gen)  # noqa: E731
    state = {"case": case}
    if case["op"] == "logp":
        rows, vocab = case["rows"], case["vocab"]
        x = randn(rows, case["stride"]).mul_(2.0)
        x[:, :vocab] -= torch.log(torch.arange(vocab, device=_DEV, dtype=torch.float32) + 2.7)
        targets = _ids(rows, vocab, 0.0, gen)
        x.scatter_add_(1, targets[:, None], 4.0 * rand(rows, 1))
        if case["banned"]:
            x.masked_fill_(rand(rows, case["stride"]) < case["banned"], -_INF)
        if case["ragged"]:
            x[3::17] = -_INF
            targets[5::11] = -100
        state.update(logits=x.to(_T[case["dtype"]])[:, :vocab], targets=targets)
        if case["grad"]:
            state.update(g=randn(rows) / rows, h=torch.full((rows,), 0.01 / rows, device=_DEV))
    elif case["op"] == "embed":
        state.update(weight=(randn(case["vocab"], case["dim"]) * 0.02).to(_T[case["weight"]]),
                     ids=_ids(case["tokens"], case["vocab"], case["padded"], gen))
    elif case["op"] == "embed_grad":
        state.update(grad=(randn(case["tokens"], case["dim"]) * 1e-3).to(_T[case["grad"]]),
                     ids=_ids(case["tokens"], case["vocab"], case["padded"], gen))
        if case["add"]:
            state["dweight"] = (randn(case["vocab"], case["dim"]) * 1e-3).to(_T[case["weight"]])
    else:
        mats, vecs = _matrices(case), _vectors(case)
        size = np.random.RandomState(seed % (1 << 31)).lognormal(math.log(1e-3), 1.0, len(mats) + len(vecs)).tolist()
        state["grads"] = [(randn(*s) * a).to(_T[case["grad"] if len(s) == 2 else "f32"]) for s, a in zip(mats + vecs, size)]
        flat, views = _flat(mats, case["out"])
        vflat, vviews = _flat(vecs, "f32")
        state.update(flat=flat, vflat=vflat, out=views + vviews)
    return state


# ------------------------------------------------------------------------------------ the plain form

def _top(x, k):
    """The k largest of each row, ties to the lowest index: one whole-number key for each value and place."""
    i = (x + 0.0).contiguous().view(torch.int32)  # -0 counts as 0
    key = torch.where(i < 0, i ^ 0x7FFFFFFF, i).long() * (1 << 32) + torch.arange(x.shape[1] - 1, -1, -1, device=x.device)
    return x.shape[1] - 1 - (key.topk(k, dim=1).values & 0xFFFFFFFF)


def _plain_logp(s):
    case = s["case"]
    x, t, k = s["logits"].float(), s["targets"], case["top"]
    y = x * case["scale"]
    m = y.amax(1, keepdim=True)
    m = torch.where(m == -_INF, 0.0, m)
    e = torch.exp(y - m)
    z = e.sum(1, keepdim=True)
    lse = m + torch.log(z)
    given = y.gather(1, t.clamp(min=0)[:, None])
    r = {"logp": torch.where(t[:, None] < 0, 0.0, torch.where(given == -_INF, -_INF, given - lse))[:, 0], "lse": lse[:, 0]}
    p = torch.where(e > 0, e / z, 0.0)
    logp = torch.where(e > 0, y - lse, 0.0)
    if case["entropy"]:
        r["entropy"] = -(p * logp).sum(1)
    if k:
        at = _top(x, k)
        alt = y.gather(1, at)
        r["top_ids"], r["top_logp"] = at.int(), torch.where(alt == -_INF, -_INF, alt - lse)
    if case["grad"]:
        g, h = torch.where(t < 0, 0.0, s["g"])[:, None], s["h"][:, None]
        d = -p * (g + h * (logp + r["entropy"][:, None]))
        live = torch.where(z > 0, g, 0.0)
        d.scatter_add_(1, t.clamp(min=0)[:, None], live)
        r["dlogits"] = (d * case["scale"]).to(s["logits"].dtype)
    return r


def _plain_embed(s):
    ids = s["ids"][:, None]
    return torch.where(ids < 0, 0.0, s["weight"][s["ids"].clamp(min=0)].float() * s["case"]["scale"]).to(_T[s["case"]["out"]])


def _plain_embed_grad(s):
    case, ids = s["case"], s["ids"]
    rows = torch.where(ids[:, None] < 0, 0.0, s["grad"].float() * case["scale"])
    total = torch.zeros(case["vocab"], case["dim"], device=ids.device).index_add_(0, ids.clamp(min=0), rows)
    if case["add"]:
        return s["dweight"].copy_(s["dweight"].float() + total)
    return total.to(_T[case["weight"]])


def _plain_clip(s):
    norms = torch.stack([g.float().square().sum() for g in s["grads"]]).sqrt()
    norm = norms.square().sum().sqrt()
    scale = (s["case"]["max_norm"] / norm).clamp(max=1.0)
    [o.copy_(g.float() * scale) for o, g in zip(s["out"], s["grads"])]
    return {"norm": norm, "scale": scale, "norms": norms, "out": s["flat"], "vectors": s["vflat"]}


# ------------------------------------------------------------------------------ the framework's calls

def _own_logp(s, dobb):
    case = s["case"]
    r = dobb.log_probs(s["logits"], s["targets"], scale=case["scale"], top_k=case["top"], entropy=case["entropy"])
    o = {"logp": r.logp, "lse": r.lse}
    if case["entropy"]:
        o["entropy"] = r.entropy
    if case["top"]:
        o["top_ids"], o["top_logp"] = r.top_ids, r.top_logp
    if case["grad"]:
        o["dlogits"] = dobb.log_probs_backward(s["logits"], s["targets"], r, s["g"], grad_entropy=s["h"])
    return o


def _own_embed(s, dobb):
    return dobb.embedding(s["weight"], s["ids"], scale=s["case"]["scale"], out_dtype=_T[s["case"]["out"]])


def _own_embed_grad(s, dobb):
    case = s["case"]
    if case["add"]:
        return dobb.embedding_backward(s["grad"], s["ids"], scale=case["scale"], out=s["dweight"], accumulate=True)
    return dobb.embedding_backward(s["grad"], s["ids"], case["vocab"], scale=case["scale"], dtype=_T[case["weight"]])


def _own_clip(s, dobb):
    r = dobb.clip_grads(s["grads"], s["case"]["max_norm"], out=s["out"])
    return {"norm": r.norm, "scale": r.scale, "norms": r.norms, "out": s["flat"], "vectors": s["vflat"]}


def run(state):
    op = state["case"]["op"]
    if own:
        import block_eigenbasis_preconditioning_gb300 as dobb
        return {"logp": _own_logp, "embed": _own_embed, "embed_grad": _own_embed_grad, "clip": _own_clip}[op](state, dobb)
    return {"logp": _plain_logp, "embed": _plain_embed, "embed_grad": _plain_embed_grad, "clip": _plain_clip}[op](state)


# ------------------------------------------------------------------------------------------ the work

def work(case):
    """Each input read once, each output written once; a float operation or two for each value and sum."""
    size = {"bf16": 2, "f32": 4}
    if case["op"] == "logp":
        n = case["rows"] * case["vocab"]
        small = case["rows"] * (8 + 4 + 4 + (4 if case["entropy"] else 0) + 8 * case["top"] + (8 if case["grad"] else 0))
        return {"bytes": n * size[case["dtype"]] * (2 if case["grad"] else 1) + small, "flops": n * (10 if case["grad"] else 4)}
    if case["op"] == "embed":
        n = case["tokens"] * case["dim"]
        seen = float((1.0 - (1.0 - _word_probs(case["vocab"])) ** case["tokens"]).sum())
        return {"bytes": seen * case["dim"] * size[case["weight"]] + n * size[case["out"]] + 8 * case["tokens"], "flops": n}
    if case["op"] == "embed_grad":
        n = case["tokens"] * (1.0 - case["padded"])
        seen = float((1.0 - (1.0 - _word_probs(case["vocab"])) ** n).sum())
        rows = 2 * seen if case["add"] else case["vocab"]
        return {"bytes": n * case["dim"] * size[case["grad"]] + rows * case["dim"] * size[case["weight"]] + 8 * case["tokens"],
                "flops": 2 * n * case["dim"]}
    n, v = (sum(math.prod(s) for s in t) for t in (_matrices(case), _vectors(case)))
    return {"bytes": n * (size[case["grad"]] + size[case["out"]]) + 8 * v, "flops": 3 * (n + v)}


# ------------------------------------------------------------------------------ the definition, 64 bits

def _exact_logp(s):
    case, k = s["case"], s["case"]["top"]
    y, t = s["logits"].double(), s["targets"]
    rows = torch.arange(len(t), device=y.device)
    best = y.sort(dim=1, descending=True, stable=True).indices[:, :k] if k else None
    y *= case["scale"]
    empty = (y > -_INF).sum(1) == 0
    lse = torch.logsumexp(y, 1)
    logs = y.sub_(torch.where(empty, 0.0, lse)[:, None])  # -inf where a token is banned
    p = logs.exp()
    entropy = -torch.special.xlogy(p, p).sum(1)
    none = t < 0
    r = {"logp": torch.where(none, 0.0, logs[rows, t.clamp(min=0)]), "lse": lse}
    if case["entropy"]:
        r["entropy"] = entropy
    if k:
        r["top_ids"], r["top_logp"] = best.int(), logs.gather(1, best)
    if case["grad"]:
        g, h = torch.where(none | empty, 0.0, s["g"].double()), s["h"].double()
        d = -h[:, None] * (torch.special.xlogy(p, p) + p * entropy[:, None]) - g[:, None] * p
        d[rows, t.clamp(min=0)] += g
        r["dlogits"] = d.mul_(case["scale"])
    return r


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "logp":
        return _exact_logp(s)
    if case["op"] == "embed":
        out = torch.zeros(case["tokens"], case["dim"], dtype=torch.float64, device=_DEV)
        real = s["ids"] >= 0
        out[real] = s["weight"].double()[s["ids"][real]].mul_(case["scale"])
        return out
    if case["op"] == "embed_grad":
        real = s["ids"] >= 0
        total = s["dweight"].double() if case["add"] else torch.zeros(case["vocab"], case["dim"], dtype=torch.float64, device=_DEV)
        return total.index_put_((s["ids"][real],), s["grad"].double()[real] * case["scale"], accumulate=True)
    norms = torch.stack([torch.linalg.vector_norm(g.double()) for g in s["grads"]])
    norm = torch.linalg.vector_norm(norms)
    scale = torch.minimum(torch.ones_like(norm), case["max_norm"] / norm)
    flat = torch.zeros(s["flat"].shape, dtype=torch.float64, device=_DEV)
    vflat = torch.zeros(s["vflat"].shape, dtype=torch.float64, device=_DEV)
    at = [o.storage_offset() for o in s["out"]]
    [(flat if g.dim() == 2 else vflat)[o:o + g.numel()].copy_(g.reshape(-1)).mul_(scale) for o, g in zip(at, s["grads"])]
    return {"norm": norm, "scale": scale, "norms": norms, "out": flat, "vectors": vflat}
