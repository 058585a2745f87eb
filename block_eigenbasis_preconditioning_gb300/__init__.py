"""Dobb optimizer step on one GB300 GPU (sm_103a CUDA kernels behind a C ABI).

"Dobb: Shard-Local Preconditioning in Block-Diagonal Eigenbases"
(arXiv 2610.39412).  `Dobb` is the optimizer object; `binding` exposes the
raw C ABI; `inputs` holds the seeded synthetic input generators.  `lm` holds
the operators at the two ends of a language model and on its gradients:
log_probs, log_probs_backward, embedding, embedding_backward, grad_norm and
clip_grads.
"""
from .binding import DobbError, load_library, library_path  # noqa: F401

_LM = ("log_probs", "log_probs_backward", "LogProbs", "embedding", "embedding_backward",
       "grad_norm", "clip_grads", "GradNorm")


def __getattr__(name):
    # the optimizer and the operators need torch; import them lazily so the
    # generators and the binding load without it
    if name == "Dobb":
        from .optimizer import Dobb
        return Dobb
    if name in _LM:
        from . import lm
        globals().update({n: getattr(lm, n) for n in _LM})
        return globals()[name]
    raise AttributeError(name)
