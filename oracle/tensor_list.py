"""Oracle: the update over a list of gradient tensors, fp64.

* the global norm (L2, L1 or largest magnitude) of ``scale * g`` and the
  coefficient ``scale * min(1, max_norm / (norm + 1e-6))``;
* clipping by that coefficient;
* Adam (Kingma & Ba) with decoupled weight decay (Loshchilov & Hutter).
"""
import numpy as np

CLIP_EPS = 1e-6


def tensor_norm(g, kind: str = "l2", scale: float = 1.0) -> float:
    a = np.abs(np.asarray(g, np.float64).reshape(-1))
    if a.size == 0:
        return 0.0
    if kind == "l2":
        return scale * float(np.sqrt(np.sum(a * a)))
    if kind == "l1":
        return scale * float(np.sum(a))
    return scale * float(np.max(a))


def grad_norm(grads, max_norm: float = np.inf, kind: str = "l2", scale: float = 1.0):
    """(norm, coefficient, each tensor's norm)."""
    each = [tensor_norm(g, kind, scale) for g in grads]
    if kind == "l2":
        norm = float(np.sqrt(np.sum(np.square(each))))
    elif kind == "l1":
        norm = float(np.sum(each))
    else:
        norm = float(np.max(each)) if each else 0.0
    if not np.isfinite(norm) or norm > float(np.finfo(np.float32).max):
        return norm, 0.0, each
    return norm, scale * min(1.0, max_norm / (norm + CLIP_EPS)), each


def clip(g, coef: float):
    g = np.asarray(g, np.float64)
    return np.zeros_like(g) if coef == 0.0 else coef * g


def adamw_step(p, g, m, v, step: int, lr: float, b1: float, b2: float, eps: float, decay: float = 0.0,
               coef: float = 1.0):
    """(p, m, v) after one step on ``coef * g``; ``step`` counts from 1."""
    p, m, v = (np.asarray(x, np.float64) for x in (p, m, v))
    g = clip(g, coef)
    m = b1 * m + (1.0 - b1) * g
    v = b2 * v + (1.0 - b2) * g * g
    mh = m / (1.0 - b1 ** step)
    vh = v / (1.0 - b2 ** step)
    return p - lr * mh / (np.sqrt(vh) + eps) - lr * decay * p, m, v
