"""What follows a gradient sync, in fp64: the global norm, clipping, AdamW.

"PyTorch DDP Deep Dive", Part 2 (after finalize_backward every rank's optimizer
applies the same update to the same averaged gradients). Plain formulas, element
by element, on one replica's tensors; bf16 inputs come as the fp32 values they
stand for. Squares of fp32 values neither overflow nor underflow in fp64.
"""
from __future__ import annotations

import math

import numpy as np

CLIP_EPS = 1e-6


def norms(grads, kind: str = "l2"):
    """(global norm, [each tensor's norm]) of a list of arrays."""
    if kind == "inf":
        each = [float(np.max(np.abs(np.asarray(g, np.float64)))) if g.size else 0.0 for g in grads]
        return (float("nan") if any(math.isnan(x) for x in each) else max(each)), each
    sums = [math.fsum(np.square(np.asarray(g, np.float64)).tolist()) if np.all(np.isfinite(g))
            else float(np.sum(np.square(np.asarray(g, np.float64)))) for g in grads]
    whole = math.fsum(sums) if all(math.isfinite(x) for x in sums) else float(np.sum(sums))
    return math.sqrt(whole), [math.sqrt(x) for x in sums]


def coefficient(norm: float, max_norm: float) -> float:
    """min(1, max_norm / (norm + 1e-6)); a NaN stays one. An infinite max_norm
    clips nothing, whatever the norm: 1."""
    if math.isnan(norm):
        return norm
    if math.isinf(max_norm):
        return 1.0
    return min(1.0, max_norm / (norm + CLIP_EPS))


def clip(grads, max_norm: float, kind: str = "l2"):
    """(norm, the scaled gradients)."""
    n, _ = norms(grads, kind)
    c = coefficient(n, max_norm)
    with np.errstate(invalid="ignore"):
        return n, [c * np.asarray(g, np.float64) for g in grads]


def adamw(w, g, m, v, step: int, lr, beta1, beta2, eps, weight_decay, c: float = 1.0):
    """One step of one tensor from `step` steps taken: (w, m, v) after it."""
    t = step + 1
    w, g, m, v = (np.asarray(x, np.float64) for x in (w, g, m, v))
    g = c * g
    m = beta1 * m + (1.0 - beta1) * g
    v = beta2 * v + (1.0 - beta2) * g * g
    m_hat = m / (1.0 - beta1 ** t)
    v_hat = v / (1.0 - beta2 ** t)
    return w - lr * weight_decay * w - lr * m_hat / (np.sqrt(v_hat) + eps), m, v
